"""Shared by the GPU tests of the layers: strided matrices with NaN around them, types, a graph's replay."""
import torch

NAN = float("nan")
DT = {0: torch.float16, 1: torch.bfloat16, 2: torch.float32}
HALF_ULP = {0: 2.0 ** -11, 1: 2.0 ** -8}
SUB = {0: 2.0 ** -25, 1: 0.0}          # half of the step below the normal range (bf16's lies below anything used here)


def rows(t, width, pad, dt, gen, scale=1.0, shift=0, offset=0.0):
    """[t, width] values in rows of width + pad elements, `shift` elements into their buffer; NaN around them."""
    buf = torch.full((t * (width + pad) + shift + 16,), NAN, dtype=dt, device="cuda")
    v = torch.as_strided(buf, (t, width), (width + pad, 1), shift)
    if t:
        v.copy_(torch.randn((t, width), generator=gen, device="cuda") * scale + offset)
    return v, buf


def outside_untouched(view, buf):
    keep = buf.clone()
    torch.as_strided(keep, view.shape, view.stride(), view.storage_offset()).fill_(NAN)
    return bool(torch.isnan(keep).all())


def assert_within(got, ref, err, ty, what=""):
    """got (16 bits) against ref (64 bits), which the unrounded result misses by at most err."""
    bad = (got.double() - ref).abs() - (err + HALF_ULP[ty] * (ref.abs() + err) + SUB[ty])
    assert not bool(torch.isnan(bad).any()) and float(bad.max()) <= 0, (what, float(bad.max()), int(bad.argmax()))


def replayed(call, outputs):
    """The outputs of `call(stream)` captured on a side stream and replayed into cleared outputs."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(side)
    for o in outputs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    return [o.clone() for o in outputs]
