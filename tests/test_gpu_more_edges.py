"""The convolution, scan, rotary and page calls where offsets pass 32 bits, on streams of their own, and two at once."""
import pytest
import torch

import test_gpu_causal_conv as conv
import test_gpu_rotary as rot
import test_gpu_selective_scan as scan
from test_gpu_pages import Both

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rp():
    import replayssm_persistent_rssm_amd as rp
    return rp


def far(t, stride):
    """t with rows `stride` elements apart."""
    room = torch.empty((t.shape[0] - 1) * stride + t[0].numel(), dtype=t.dtype, device="cuda")
    v = room.as_strided(t.shape, (stride,) + t.stride()[1:])
    v.copy_(t)
    return v


@pytest.mark.parametrize("step", [False, True])
def test_convolution_rows_and_slots_far_apart(rp, step):
    p = conv.inputs([1] * 7 if step else [3, 0, 9], 72, 4, "bf16", seed=1, extra=6)
    conv.check(rp, p, x=far(p["x"], 2 ** 28), y=far(torch.full_like(p["x"], float("nan")), 2 ** 28 + 8),
               state=far(p["state"], 2 ** 28), step=step)


@pytest.mark.parametrize("step", [False, True])
def test_scan_rows_and_slots_far_apart(rp, step):
    p = scan.inputs([1] * 140 if step else [100, 0, 170], 64, it="bf16", seed=2, extra=6)
    d = scan.on_device(p)
    for k in ("x", "dt", "z"):
        d[k] = far(p[k], 2 ** 24)
    scan.check(rp, p, d=d, y=far(torch.full_like(p["x"], float("nan")), 2 ** 24), st=far(p["state"], 2 ** 25 if step else 2 ** 28), step=step)


def test_stretches_far_apart(rp):
    p = scan.inputs([700], 16, it="bf16", seed=3)
    d = scan.on_device(p)
    for k in ("x", "dt", "B", "C"):
        d[k] = far(p[k], 2 ** 22)
    scan.check(rp, p, d=d, use=("D", "bias"))


def test_rotary_pages_and_rows_far_apart(rp):
    p = rot.inputs([9, 3], [60, 3], 4, 2, 64, 64, seed=4)
    d = {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)}
    d["kc"], d["vc"] = far(p["kc"], 2 ** 29), far(p["vc"], 2 ** 29)
    d["q"], d["k"], d["v"] = far(p["q"], 2 ** 28), far(p["k"], 2 ** 27), far(p["v"], 2 ** 27)
    rot.check(rp, p, d=d, out=far(torch.full_like(p["q"], float("nan")), 2 ** 28 + 8))


def test_pages_far_apart(rp):
    """Pages half a gigabyte apart: the bytes of forks and moves are looked at where they lie."""
    b = Both(rp, rows=4, most=3, pages=12, page=16, caches=1, wide=64)
    room = torch.zeros(11 * 2 ** 29 + 1024, dtype=torch.uint8, device="cuda")
    far_cache = room.as_strided((12, 1024), (2 ** 29, 1))
    far_cache.copy_(b.room[0])
    b.ptrs = torch.tensor([room.data_ptr()], dtype=torch.int64, device="cuda")
    b.caches["page_stride"] = 2 ** 29
    b.dev = far_cache[None]
    b.extend([0, 1], [40, 48])
    b.fork([0, 1], [2, 3], [37, 20])
    b.release([0])
    b.compact()
    src, dst = b.i32([1, 2]), b.i32([10, 11])
    rp.rssm_page_copy(b.ptrs, src, dst, num_pages=12, page_bytes=1024, page_stride=2 ** 29)
    b.room[0, 10:12] = b.room[0, 1:3]
    assert torch.equal(b.dev.cpu(), b.room)


def test_on_a_stream_of_its_own(rp):
    """Given by stream=, with and without a workspace: ordered after what that stream waits for, results as on the current one."""
    s = torch.cuda.Stream()
    p = conv.inputs([30, 1, 9], 128, 4, "bf16", seed=5)
    d = {k: v.cuda() for k, v in p.items() if torch.is_tensor(v)}
    ys, sts = [torch.zeros_like(d["x"]) for _ in range(2)], [d["state"].clone() for _ in range(2)]
    r = rot.inputs([5, 2], [40, 2], 4, 2, 64, 64, seed=6)
    e = {k: v.cuda() for k, v in r.items() if torch.is_tensor(v)}
    qs, ks, vs = ([t.clone() for _ in range(2)] for t in (e["q"], e["kc"], e["vc"]))
    pools = [Both(rp, rows=4, most=6, pages=30, page=16) for _ in range(2)]
    st = [torch.zeros(2, dtype=torch.int32, device="cuda") for _ in range(2)]
    live = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
    rows, more, add = (pools[0].i32(v) for v in ([0, 1], [2, 3], [50, 20]))
    s.wait_stream(torch.cuda.current_stream())
    for i, stream in enumerate((None, s)):
        b = pools[i]
        pool = (b.table, b.kv, b.ref)
        rp.rssm_causal_conv(d["x"], d["weight"], ys[i], sts[i], d["slots"], d["starts"], stream=stream)
        rp.rssm_causal_conv_step(ys[i][:3], d["weight"], ys[i][:3], sts[i], d["slots"], stream=stream)
        rp.rssm_rotary_append(qs[i], qs[i], ks[i], vs[i], e["k"], e["v"], e["table"], e["starts"], e["kv"], e["freq"], stream=stream)
        rp.rssm_page_extend(*pool, rows, add, st[i], page_size=16, stream=stream)
        rp.rssm_page_fork(b.ptrs, *pool, rows, more, st[i], token_bytes=32, stream=stream, **b.caches)
        rp.rssm_page_release(*pool, rows, page_size=16, stream=stream)
        rp.rssm_page_compact(b.ptrs, *pool, live[i], stream=stream, **b.caches)
    torch.cuda.synchronize()
    for a in (ys, sts, qs, ks, vs, st, live, [b.table for b in pools], [b.kv for b in pools], [b.ref for b in pools], [b.dev for b in pools]):
        assert torch.equal(*a)
    assert live[0].item() > 0


def test_two_scans_at_once(rp):
    """Side by side on two streams, each with stretches and a workspace of its own."""
    p = [scan.inputs([900, 40], 256, seed=7 + i) for i in range(2)]
    d = [scan.on_device(q) for q in p]
    want = []
    for q, e in zip(p, d):
        y, st = torch.zeros_like(e["x"]), e["state"].clone()
        scan.call(rp, q, e, y, st)
        want.append((y, st))
    got = [(torch.zeros_like(e["x"]), e["state"].clone()) for e in d]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s, q, e, (y, st) in zip(streams, p, d, got):
            with torch.cuda.stream(s):
                st.copy_(e["state"])
                scan.call(rp, q, e, y, st)
    torch.cuda.synchronize()
    for (a, b), (c, e) in zip(want, got):
        assert torch.equal(a, c) and torch.equal(b, e)


def test_refusals_of_the_binding(rp):
    """Device tensors of the wrong kind: named, nothing enqueued."""
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")      # noqa: E731
    i = lambda *s: z(*s, dtype=torch.int32)                                              # noqa: E731
    good = dict(x=z(3, 16), weight=z(4, 16), y=z(3, 16), state=z(2, 3, 16), slots=i(1), seq_start=i(2))
    for name, bad in (("x", z(16, 3).T), ("weight", z(4, 8)), ("y", z(3, 16, dtype=torch.float16)), ("state", z(2, 2, 16)), ("slots", z(1)),
                      ("seq_start", i(1)), ("weight", z(4, 16).cpu())):
        with pytest.raises(ValueError, match=name):
            rp.rssm_causal_conv(**{**good, name: bad})
    with pytest.raises(rp.RssmError, match="y may not be x"):
        rp.rssm_causal_conv(good["x"], good["weight"], good["x"], good["state"], good["slots"], good["seq_start"])
    good = dict(state=z(2, 16, 16), A=z(16, 16), x=z(3, 16), B=z(3, 1, 16), C=z(3, 1, 16), dt=z(3, 16), y=z(3, 16), slots=i(1), seq_start=i(2))
    for name, bad in (("A", z(16, 8)), ("B", z(3, 1, 32)), ("C", z(2, 1, 16)), ("dt", z(3, 16, dtype=torch.float16)), ("y", z(3, 8)), ("state", z(2, 16, 32)[:, :, ::2]),
                      ("slots", i(2, 1)), ("seq_start", i(3))):
        with pytest.raises(ValueError, match=name):
            rp.rssm_selective_scan(**{**good, name: bad}, max_seq_len=3)
    with pytest.raises(rp.RssmError, match="workspace"):
        big = {**good, "x": z(2000, 16), "dt": z(2000, 16), "y": z(2000, 16), "B": z(2000, 1, 16), "C": z(2000, 1, 16)}
        rp.rssm_selective_scan(**big, max_seq_len=2000, workspace=z(16, dtype=torch.uint8))
    kc, t, s, k, q, f = z(4, 16, 2, 64), i(1, 4), i(2), i(1), z(1, 4, 64), z(32)
    for name, args in (("v_cache", (q, q, kc, z(4, 16, 2, 128), z(1, 2, 64), z(1, 2, 64), t, s, k, f)),
                       ("k_new", (q, q, kc, kc, z(1, 3, 64), z(1, 2, 64), t, s, k, f)), ("q_out", (q, z(2, 4, 64), kc, kc, z(1, 2, 64), z(1, 2, 64), t, s, k, f)),
                       ("inv_freq", (q, q, kc, kc, z(1, 2, 64), z(1, 2, 64), t, s, k, z(4, 8)))):
        with pytest.raises(ValueError, match=name):
            rp.rssm_rotary_append(*args)
    with pytest.raises(rp.RssmError, match="rot_dim"):
        rp.rssm_rotary_append(q, q, kc, kc, z(1, 2, 64), z(1, 2, 64), t, s, k, z(36))
    with pytest.raises(ValueError, match="positions"):
        rp.rssm_rotary_append(q, q, None, None, None, None, None, None, None, f)
    table, kv, refs, st = i(2, 4), i(2), i(8), i(1)
    for name, args in (("kv_len", (table, i(3), refs, i(1), i(1), st)), ("page_ref", (table, kv, z(8), i(1), i(1), st)), ("rows", (table, kv, refs, z(1), i(1), st)),
                       ("add", (table, kv, refs, i(1), i(2), st)), ("status", (table, kv, refs, i(1), i(1), i(2))), ("page_table", (i(4, 2).T, kv, refs, i(1), i(1), st))):
        with pytest.raises(ValueError, match=name):
            rp.rssm_page_extend(*args, page_size=16)
    ptrs = z(1, dtype=torch.int64)
    with pytest.raises(rp.RssmError, match="token_bytes"):
        rp.rssm_page_fork(ptrs, table, kv, refs, i(1), i(1), st, page_size=16, page_bytes=1024, token_bytes=32)
    with pytest.raises(rp.RssmError, match="page_bytes"):
        rp.rssm_page_compact(ptrs, table, kv, refs, i(1), page_size=16, page_bytes=1000)
    with pytest.raises(rp.RssmError, match="workspace"):
        rp.rssm_page_extend(table, kv, refs, i(1), i(1), st, page_size=16, workspace=z(16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="cache_ptrs"):
        rp.rssm_page_copy(i(1), i(1), i(1), num_pages=8, page_bytes=1024)
    assert not table.any() and not kv.any() and not refs.any()
