"""What rssm_rotary_append does not turn is copied bit by bit: values, and heads past rot_dim."""
import pytest
import torch

import test_gpu_rotary as rot

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rp():
    import replayssm_persistent_rssm_amd as rp
    return rp


def bits(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("it", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,turned,tokens", [(64, 16, 70), (128, 64, 70), (128, 128, 70), (64, 32, 4200)])
def test_copies_keep_every_bit(rp, it, inter, D, turned, tokens):
    """Any pattern of bits: signalling and quiet NaN, infinities, numbers below the normal ones.  In place too; many tokens
    take the form of one wavefront a token."""
    p = rot.inputs([tokens, 3], [tokens, 20], 4, 2, D, turned, it, seed=D + turned)
    g = torch.Generator().manual_seed(turned)
    for k in ("q", "k", "v"):
        b = bits(p[k])
        part = b if k == "v" else b[..., turned:]
        part.copy_(torch.randint(-2 ** 31, 2 ** 31, part.shape, generator=g).to(b.dtype))
    d = {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)}
    kc, vc, out = p["kc"].clone(), p["vc"].clone(), torch.empty_like(d["q"])
    rp.rssm_rotary_append(d["q"], out, d["kc"], d["vc"], d["k"], d["v"], d["table"], d["starts"], d["kv"], d["freq"], interleaved=inter)
    assert torch.equal(bits(out.cpu())[..., turned:], bits(p["q"])[..., turned:])
    page = p["page"]
    at = p["pos"].long()
    pages = p["table"][torch.tensor(p["seq"]), at // page].long()
    bits(kc)[pages, at % page], bits(vc)[pages, at % page] = bits(p["k"]), bits(p["v"])
    assert torch.equal(bits(d["vc"].cpu()), bits(vc))
    assert torch.equal(bits(d["kc"].cpu())[..., turned:], bits(kc)[..., turned:])
    rp.rssm_rotary_append(d["q"], d["q"], d["kc"], d["vc"], d["k"], d["v"], d["table"], d["starts"], d["kv"], d["freq"], interleaved=inter)
    assert torch.equal(bits(d["q"]), bits(out))
