"""The workspace that the embedding's gradient asks for, against the bound that its header states."""
import pytest

SIZES = [(T, D, V) for T in (*range(1, 10), 31, 509, 1024, 2433, 8192, 8193, 38912, 65536, 65537, 70000, 10 ** 6, 5 * 10 ** 7)
         for D in (1, 8, 9, 40, 250, 257, 2048, 8192) for V in (1, 511, 512, 44629, 1 << 20, 1 << 30)]


def stated(T, D):
    return 2 * (T + 3) * (D + 23) + 17408


@pytest.mark.parametrize("T", sorted({s[0] for s in SIZES}))
def test_stated_bound(zlib, T):
    for t, D, V in SIZES:
        if t == T:
            assert zlib.zero_embed_workspace(T, D, V) <= stated(T, D), (T, D, V)


def test_nothing_for_no_tokens(zlib):
    assert zlib.zero_embed_workspace(0, 64, 100) == 0


def test_many_tokens_need_less(zlib):
    """The header's "about an eighth": chunks of 32 tokens and more in place of 4."""
    for T, D in ((65536, 2048), (200000, 1024), (10 ** 6, 2048)):
        assert zlib.zero_embed_workspace(T, D, 50000) <= stated(T, D) / 7
