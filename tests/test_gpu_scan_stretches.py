"""The selective scan with its token axis in stretches: resumed prompts, last stretches of one token, more workgroups than the
device holds at once, channel blocks (of 64) in numbers that 8 does not divide."""
import pytest
import torch

import more_operators_ref as ref
import test_gpu_selective_scan as scan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rp():
    import replayssm_persistent_rssm_amd as rp
    return rp


def workspace(rp, p, d, most):
    return rp.rssm_selective_scan_workspace(d["state"], *(d[k] for k in ("A", "x", "B", "C", "dt", "z", "slots", "starts")), max_seq_len=most)


@pytest.mark.parametrize("lens,Ch,n,it,st", [
    ([1025, 1025], 2560, 16, "bf16", "f32"),      # 17 stretches of 64 tokens, 1,360 workgroups
    ([2001], 1032, 16, "f16", "bf16"),            # 26 of 80
    ([385, 97, 385], 264, 32, "bf16", "f16"),     # 9 of 48
    ([385], 1032, 64, "f32", "f32"),              # 9 of 48
])
def test_a_last_stretch_of_one_token(rp, lens, Ch, n, it, st):
    """All resumed from the pool: every stretch starts from what the slot held before the call."""
    p = scan.inputs(lens, Ch, n, 1, it, st, seed=n + Ch)
    d = scan.on_device(p)
    assert workspace(rp, p, d, max(lens)) > 0
    y, pool = scan.check(rp, p, use=("D", "bias", "z"), d=d)
    for _ in range(3):
        again, st2 = torch.empty_like(y), d["state"].clone()
        scan.call(rp, p, d, again, st2, use=("D", "bias", "z"))
        assert torch.equal(again, y) and torch.equal(st2, pool)


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("st", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,G", [(16, 1), (32, 4), (64, 2)])
def test_every_type_and_number_of_states(rp, it, st, n, G):
    """Resumed and new prompts, skipped slots, ends at, before and after the borders; all optional inputs and none."""
    p = scan.inputs([385, 48, 49, 0, 47, 96, 330, 1], 192, n, G, it, st, seed=n, slots=[3, 0, 7, 5, 2, 9, -1, 8])
    assert workspace(rp, p, scan.on_device(p), 385) > 0
    scan.check(rp, p)
    scan.check(rp, p, use=("load",))


@pytest.mark.parametrize("it,st,n", [("bf16", "f32", 16), ("f16", "bf16", 32), ("f32", "f16", 64)])
def test_the_start_goes_through_the_workspace(rp, it, st, n):
    """The first launch leaves it in the entry of the sequence's last stretch (of 9, 48 tokens each), zeros where
    load_state is 0; sequences of one stretch, and of none, have no entry."""
    lens, last = [385, 97, 40, 385, 0, 49, 96], [8, 2, 0, 8, 0, 1, 1]
    p = scan.inputs(lens, 40, n, 1, it, st, seed=n)
    d = scan.on_device(p)
    need = workspace(rp, p, d, 385)
    assert need == 7 * 9 * 40 * (n + 1) * 4
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    y, pool = torch.empty_like(d["x"]), d["state"].clone()
    scan.call(rp, p, d, y, pool, ws=ws)
    ends = ws.view(torch.float32)[:7 * 9 * 40 * n].view(7, 9, 40, n).cpu()
    for s, k in enumerate(last):
        if k > 0:
            start = p["state"][int(p["slots"][s])].float() if int(p["load"][s]) else torch.zeros(40, n)
            assert torch.equal(ends[s, k], start), s
        else:
            assert torch.isnan(ends[s]).all(), s
    assert set(p["load"][i].item() for i, k in enumerate(last) if k) == {0, 1}
    want, m, state, sm = ref.scan(p["state"], p["A"], p["x"], p["B"], p["C"], p["dt"], p["slots"], p["seqs"], D=p["D"], bias=p["bias"],
                                  z=p["z"], load=p["load"])
    ref.check(y, want, ref.scan_bound(want, m, y.dtype, ref.scan_chain(385, n)), "y")
    ref.check(pool, state, ref.scan_bound(state, sm, pool.dtype, ref.scan_chain(385, n)), "state")


@pytest.mark.parametrize("n", [16, 32, 64])
def test_nothing_grows_to_nothing(rp, n):
    """States that start at zero and have not been written to yet stay zero, however far a stretch would have made them grow
    (exp(96) here, past fp32)."""
    p = scan.inputs([700, 690], 64, n, 1, "f32", "f32", seed=n)
    d = scan.on_device(p)
    assert workspace(rp, p, d, 700) > 0
    p["A"][:, 3], p["A"][:, n - 1] = 1.0, 0.5
    p["dt"][:] = 2.0
    p["load"][:] = 0
    p["x"][:690], p["x"][700:1380] = 0.0, 0.0
    scan.check(rp, p, use=("D", "z", "load"), softplus=False)
