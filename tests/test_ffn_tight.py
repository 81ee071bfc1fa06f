"""That the tight checks of the 4-bit and gated products can fail: mistakes planted in the reference, on the CPU."""
import numpy as np
import pytest

from tests.ffn_exact_cases import in_use, once, result, tight, whole

torch = pytest.importorskip("torch")

KINDS = ["linear", "gated", "grouped", "grouped_gated"]


def case(make, kind, group, d_in, rank=0, **kw):
    return make(kind, group, np.arange(24) % 2, 2, d_in, 96, rank, **kw)


def with_scales(c, change):
    """Every weight of the case with its group scales changed."""
    return {col: [q.double() * change(s).double().repeat_interleave(c.group, 1) for _, q, s in c.W[col]] for col in c.cols}


bf16 = lambda t: t.to(torch.bfloat16).to(t.dtype)  # noqa: E731
cut = lambda t: (t.float().view(torch.int32) & -65536).view(torch.float32).to(t.dtype)  # noqa: E731


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group,d_in", [(32, 384), (128, 384), (128, 1152), (64, 2176), (128, 8320)])
def test_tight_passes_a_rounding_and_fails_mistakes(kind, group, d_in):
    c = case(in_use, kind, group, d_in, 8 if kind in ("linear", "gated") else 0)
    ref, on = result(c)
    assert bool(on.all())
    assert tight(ref.float().to(torch.bfloat16), ref)
    assert tight((ref * (1 + 2.0 ** -13)).to(torch.bfloat16), ref)  # a slip of 1/32 of a step
    wrong = {
        "scales in bf16": result(c, W=with_scales(c, bf16))[0],
        "a gain of 0.3%": ref * 1.003,
        "a gain of 0.3% of one projection": result(c, lambda col, y: y * (1.003 if col == c.cols[-1] else 1))[0],
        "sums cut to bf16": result(c, lambda col, y: cut(y))[0],
    }
    if c.is_gated:
        wrong["g and u rounded to bf16"] = result(c, lambda col, y: bf16(y))[0]
        wrong["g alone rounded to bf16"] = result(c, lambda col, y: bf16(y) if col == "gate" else y)[0]
    for what, y in wrong.items():
        assert not tight(y.to(torch.bfloat16), ref), what


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group,d_in", [(32, 384), (128, 1152), (64, 2176)])
def test_exact_cases_fail_mistakes(kind, group, d_in):
    c = case(whole, kind, group, d_in)
    want, on = once(c)
    product = lambda W={}, f=lambda y: y: torch.stack([f(c.sums(col, W.get(col))[0]).float() for col in c.cols]).prod(0)  # noqa: E731
    assert torch.equal(product().to(torch.bfloat16), want)
    assert not torch.equal(product(with_scales(c, bf16)).to(torch.bfloat16), want)
    if c.is_gated:
        assert not torch.equal(product(f=bf16).to(torch.bfloat16), want)
    else:
        assert not torch.equal(cut(product()).to(torch.bfloat16), want)


@pytest.mark.parametrize("group,rank", [(32, 40), (64, 5), (128, 16), (0, 16)])
@pytest.mark.parametrize("kind", ["linear", "gated"])
def test_exact_cases_fail_a_v_of_16_bits(kind, group, rank):
    if kind == "linear" and not group:
        return  # no such call
    c = case(whole, kind, group, 1152, rank)
    want, _ = once(c)

    def two_pieces(t):  # v scaled, as the sum of two bf16 values
        hi = bf16(t.float())
        return (hi + bf16(t.float() - hi)).double()

    def sums(col):
        x, y = c.x.double(), c.x.double() @ c.W[col][0][0].t()
        for s in range(2):
            at = c.ids == s
            y[at] += two_pieces(c.scale[col][s] * (x[at] @ c.A[col][s].double().t())) @ c.B[col][s].double().t()
        return y.float()

    got = torch.stack([sums(col) for col in c.cols]).prod(0).to(torch.bfloat16)
    assert float((got != want).float().mean()) > 0.01
