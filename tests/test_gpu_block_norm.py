"""rssm_block_norm against its formulas in 64 bits."""
import math

import pytest
import torch

import operators_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rp():
    import replayssm_persistent_rssm_amd as rp
    return rp


def inputs(R, C, it, rt, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)          # noqa: E731
    return dict(y=rn(R, C).to(ref.DT[it]), z=rn(R, C).to(ref.DT[it]), residual=(2 * rn(R, C)).to(ref.DT[rt]),
                post=1 + 0.1 * rn(C), pre=1 + 0.1 * rn(C), cs=0.5 + 0.1 * rn(C))


def check(rp, p, *, use=("z", "post", "pre", "cs"), groups=1, rs=0.7, eps=1e-5, normed=True):
    c = lambda k: p[k].cuda() if k in use else None      # noqa: E731
    y, res = p["y"].cuda(), p["residual"].cuda()
    ro = torch.full_like(res, math.nan)
    n = torch.full_like(y, math.nan) if normed else None
    rp.rssm_block_norm(y, res, ro, n, z=c("z"), post_weight=c("post"), pre_weight=c("pre"), channel_scale=c("cs"),
                       residual_scale=rs, groups=groups, eps=eps)
    h = lambda k: p[k] if k in use else None             # noqa: E731
    r, rm, nn, nm = ref.block_norm(p["y"], p["residual"], z=h("z"), post=h("post"), pre=h("pre"), cs=h("cs"), rs=rs,
                                   groups=groups, eps=eps)
    ref.check(ro, r, ref.norm_bound(r, rm, ro.dtype), "residual")
    if normed:
        ref.check(n, nn, ref.norm_bound(nn, nm, n.dtype), "normed")
    assert torch.equal(res.cpu(), p["residual"]) and torch.equal(y.cpu(), p["y"])


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C,groups", [(8, 1), (1032, 1), (2048, 8), (4104, 3), (9000, 125), (16384, 2)])
def test_types_and_widths(rp, it, rt, C, groups):
    check(rp, inputs(5, C, it, rt, seed=C), groups=groups)


@pytest.mark.parametrize("use", [(), ("z",), ("post",), ("pre", "cs"), ("z", "post", "pre")])
def test_optional_inputs(rp, use):
    check(rp, inputs(3, 512, "bf16", "f32", seed=1), use=use)
    check(rp, inputs(3, 512, "f16", "f16", seed=2), use=tuple(k for k in use if k != "pre"), normed=False)


def test_one_row_and_many(rp):
    check(rp, inputs(1, 256, "bf16", "f32", seed=3))
    check(rp, inputs(3001, 64, "bf16", "f32", seed=4), groups=4)


def test_extreme_gates(rp):
    p = inputs(4, 128, "f32", "f32", seed=5)
    p["z"][:2] = torch.tensor([-1e4, 1e4]).repeat_interleave(1)[:, None]
    check(rp, p)


def test_in_place(rp):
    p = inputs(6, 1000, "bf16", "f32", seed=6)
    y, res = p["y"].cuda(), p["residual"].cuda()
    rp.rssm_block_norm(y, res, res, y, post_weight=p["post"].cuda(), pre_weight=p["pre"].cuda())
    r, rm, n, nm = ref.block_norm(p["y"], p["residual"], post=p["post"], pre=p["pre"])
    ref.check(res, r, ref.norm_bound(r, rm, res.dtype), "residual")
    ref.check(y, n, ref.norm_bound(n, nm, y.dtype), "normed")


def test_strided_rows_and_nonfinite_row(rp):
    p = inputs(4, 264, "bf16", "bf16", seed=7)
    wide = torch.full((4, 400), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:272] = p["y"].cuda()
    res = torch.full((4, 272), math.nan, dtype=torch.bfloat16, device="cuda")
    res[:, :264] = p["residual"].cuda()
    out = torch.zeros(4, 320, dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(4, 288, dtype=torch.bfloat16, device="cuda")
    wide[2, 8] = math.inf
    rp.rssm_block_norm(wide[:, 8:272], res[:, :264], out[:, :264], n[:, :264])
    r, rm, nn, nm = ref.block_norm(p["y"], p["residual"])
    rows = [0, 1, 3]           # row 2 has an infinity; no other row sees it
    ref.check(out[rows, :264], r[rows], ref.norm_bound(r, rm, out.dtype)[rows], "residual")
    ref.check(n[rows, :264], nn[rows], ref.norm_bound(nn, nm, n.dtype)[rows], "normed")
    assert (out[:, 264:] == 0).all() and (n[:, 264:] == 0).all()


def test_no_rows(rp):
    e = torch.empty(0, 64, device="cuda")
    rp.rssm_block_norm(e, e, e, e)
