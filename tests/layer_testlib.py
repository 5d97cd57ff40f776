"""Helpers of the tests of the operators around the gated delta rule: 64-bit
definitions in torch on the GPU (written from the formulas, independent of the
library), tolerances counted in half-steps of the output type, and buffers with
guard bands."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24  # half a step of fp32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def unit(g, *shape, dtype=torch.float32):
    x = torch.randn(shape, generator=g, device="cuda")
    return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-30)).to(dtype)


def assert_within(got, want, tol, what=""):
    """|got - want| <= tol element by element (NaN only where the definition has one)."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(got.isnan(), want.isnan()), f"{what}: NaN in other places"
    err = (got - want).abs().nan_to_num(0.0)
    tol = (torch.as_tensor(tol, device=err.device, dtype=torch.float64) + 0.0 * err).nan_to_num(0.0)
    bad = err > tol
    if bad.any():
        i = int((err - tol).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance; worst at flat {i}: got "
                             f"{got.flatten()[i].item():.8g}, want {want.flatten()[i].item():.8g}, "
                             f"tol {tol.flatten()[i].item():.3g}")


class Guarded:
    """A tensor between two bands of a byte pattern; check() says whether the bands are untouched."""
    BAND, PATTERN = 4096, 0xA5

    def __init__(self, shape, dtype, offset=0):
        n = 1
        for d in shape:
            n *= d
        es = torch.empty((), dtype=dtype).element_size()
        self.lo, self.n = self.BAND + offset * es, n * es
        self.raw = torch.full((self.lo + self.n + self.BAND,), self.PATTERN, dtype=torch.uint8, device="cuda")
        self.t = self.raw[self.lo:self.lo + self.n].view(dtype).view(shape)

    def check(self, what=""):
        torch.cuda.synchronize()
        assert bool((self.raw[:self.lo] == self.PATTERN).all()), f"{what}: written before the buffer"
        assert bool((self.raw[self.lo + self.n:] == self.PATTERN).all()), f"{what}: written behind the buffer"


def captured(fn, warm=True):
    """A CUDA graph of fn() (called once on a side stream first); returns (graph, fn's last result)."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    if warm:
        with torch.cuda.stream(s):
            fn()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = fn()
    return g, r
