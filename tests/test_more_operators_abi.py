"""Host-side refusals of the causal convolution, selective scan, rotary and page-pool calls: bad arguments return
before any HIP call, so nothing here needs a GPU or launches a kernel."""
import ctypes
import math
import os
import re

import pytest
import torch

from test_operators_abi import fake


@pytest.fixture(scope="module")
def rp():
    import replayssm_persistent_rssm_amd as rp
    return rp


def build(cls, base, kw):
    return cls(**{**base, **kw})


CONV = dict(num_seqs=4, num_tokens=100, channels=1024, width=4, num_slots=8, pad_slot_id=-1, dtype=1, silu=1,
            state_slot_stride=3 * 1024, x_token_stride=1024, y_token_stride=1024)
SCAN = dict(num_seqs=4, num_tokens=100, channels=1024, groups=2, dstate=16, num_slots=8, pad_slot_id=-1, max_seq_len=40,
            state_dtype=0, input_dtype=1, dt_softplus=1, reserved=0, state_slot_stride=1024 * 16, x_token_stride=1024,
            dt_token_stride=1024, B_token_stride=32, C_token_stride=32, z_token_stride=1024, y_token_stride=1024, workspace_bytes=0)
ROT = dict(num_seqs=2, num_tokens=10, num_q_heads=8, num_kv_heads=2, head_dim=128, rot_dim=128, interleaved=0, page_size=16,
           num_pages=100, max_pages=50, dtype=1, factor=1.0, page_stride=16 * 256, row_stride=256, head_stride=128,
           q_token_stride=1024, q_out_token_stride=1024, k_token_stride=256, v_token_stride=256, table_stride=50)
PAGES = dict(num_items=3, num_rows=8, max_pages=10, num_pages=100, page_size=16, num_caches=4, table_stride=10, page_bytes=16 * 64,
             page_stride=16 * 64, token_bytes=64, workspace_bytes=1 << 20)

BAD_CONV = [
    (dict(num_seqs=-1), 1, "num_seqs"), (dict(num_tokens=-1), 1, "num_tokens"), (dict(channels=0), 1, "channels"),
    (dict(channels=1020), 1, "channels"), (dict(channels=2 ** 20 + 8), 1, "channels"), (dict(width=1), 2, "width=1"),
    (dict(width=5), 2, "width=5"), (dict(num_slots=0), 1, "num_slots"), (dict(dtype=9), 1, "dtype"),
    (dict(dtype=3), 2, "f32, bf16 or f16"), (dict(silu=2), 1, "silu"), (dict(state_slot_stride=3 * 1024 - 8), 1, "state_slot_stride"),
    (dict(x_token_stride=1016), 1, "x_token_stride"), (dict(y_token_stride=1028), 1, "16 bytes"),
    (dict(x_token_stride=2 ** 32), 1, "2^31"),
]
BAD_SCAN = [
    (dict(num_seqs=-1), 1, "num_seqs"), (dict(num_tokens=-1), 1, "num_tokens"), (dict(channels=4), 1, "channels"),
    (dict(channels=1020), 1, "channels"), (dict(groups=0), 1, "groups"), (dict(groups=3), 1, "groups"), (dict(groups=128), 1, "groups"),
    (dict(dstate=8), 2, "dstate=8"), (dict(dstate=128), 2, "dstate=128"), (dict(num_slots=0), 1, "num_slots"),
    (dict(max_seq_len=-1), 1, "max_seq_len"), (dict(max_seq_len=2 ** 30 + 1), 1, "max_seq_len"), (dict(dt_softplus=2), 1, "dt_softplus"),
    (dict(reserved=1), 1, "reserved"), (dict(state_dtype=9), 1, "dtype"), (dict(state_dtype=3), 2, "f32, bf16 or f16"),
    (dict(input_dtype=4), 2, "f32, bf16 or f16"), (dict(state_slot_stride=100), 1, "state_slot_stride"),
    (dict(state_slot_stride=1024 * 16 + 2), 1, "16 bytes"), (dict(x_token_stride=8), 1, "x_token_stride"),
    (dict(dt_token_stride=1028), 1, "dt_token_stride"), (dict(B_token_stride=24), 1, "B_token_stride"),
    (dict(C_token_stride=36), 1, "C_token_stride"), (dict(z_token_stride=0), 1, "z_token_stride"),
    (dict(y_token_stride=2 ** 32), 1, "y_token_stride"), (dict(workspace_bytes=-1), 1, "workspace_bytes"),
    (dict(num_slots=2 ** 31 - 1, state_slot_stride=2 ** 44), 1, "2^46"),
]
BAD_ROT = [
    (dict(num_seqs=-1), 1, "num_seqs"), (dict(num_tokens=-1), 1, "num_tokens"), (dict(num_tokens=2 ** 24), 1, "num_tokens"),
    (dict(num_q_heads=-1), 1, "num_q_heads"), (dict(num_kv_heads=5000), 1, "num_kv_heads"), (dict(dtype=9), 1, "dtype"),
    (dict(dtype=4), 2, "f32, bf16 or f16"), (dict(head_dim=96), 2, "head_dim=96"), (dict(rot_dim=0), 1, "rot_dim"),
    (dict(rot_dim=24), 1, "rot_dim"), (dict(rot_dim=144), 1, "rot_dim"), (dict(interleaved=2), 1, "interleaved"),
    (dict(factor=math.nan), 1, "factor"), (dict(factor=math.inf), 1, "factor"), (dict(q_token_stride=1016), 1, "q_token_stride"),
    (dict(q_out_token_stride=1028), 1, "q_out_token_stride"), (dict(page_size=0), 1, "page_size"), (dict(num_pages=0), 1, "num_pages"),
    (dict(max_pages=0), 1, "max_pages"), (dict(table_stride=49), 1, "table_stride"), (dict(page_stride=64), 1, "page_stride"),
    (dict(row_stride=260), 1, "row_stride"), (dict(head_stride=0), 1, "head_stride"), (dict(k_token_stride=248), 1, "k_token_stride"),
    (dict(v_token_stride=252), 1, "v_token_stride"),
]
EVERY_POOL = [(dict(num_pages=0), 1, "num_pages"), (dict(num_pages=2 ** 30 + 1), 1, "num_pages"), (dict(workspace_bytes=-1), 1, "workspace_bytes")]
ITEMS = [(dict(num_items=-1), 1, "num_items"), (dict(num_items=2 ** 20 + 1), 1, "num_items")]
ROWS = [(dict(num_rows=0), 1, "num_rows"), (dict(num_rows=2 ** 20 + 1), 1, "num_rows"), (dict(max_pages=0), 1, "max_pages"),
        (dict(page_size=0), 1, "page_size"), (dict(table_stride=9), 1, "table_stride")]
CACHES = [(dict(num_caches=-1), 1, "num_caches"), (dict(num_caches=65536), 1, "num_caches"), (dict(page_bytes=0), 1, "page_bytes"),
          (dict(page_bytes=1032, page_stride=2048), 1, "page_bytes"), (dict(page_stride=1008), 1, "page_stride"),
          (dict(page_stride=1032), 1, "page_stride"), (dict(page_stride=2 ** 45), 1, "page_stride")]
FORK = [(dict(token_bytes=-16), 1, "token_bytes"), (dict(token_bytes=32), 1, "token_bytes"), (dict(token_bytes=8), 1, "token_bytes")]
POOL_CALLS = {"rssm_page_extend": EVERY_POOL + ITEMS + ROWS, "rssm_page_fork": EVERY_POOL + ITEMS + ROWS + CACHES + FORK,
              "rssm_page_release": EVERY_POOL + ITEMS + ROWS, "rssm_page_compact": EVERY_POOL + ROWS + CACHES,
              "rssm_page_copy": EVERY_POOL + ITEMS + CACHES}


def refused(rp, name, desc, tab, status, text):
    assert getattr(rp.lib(), name)(ctypes.byref(desc), ctypes.byref(tab), None) == status
    assert text in rp.rssm_last_error(), rp.rssm_last_error()


@pytest.mark.parametrize("kw,status,text", BAD_CONV)
def test_conv_scalars(rp, kw, status, text):
    for name in ("rssm_causal_conv", "rssm_causal_conv_step"):
        d = build(rp.RssmConvDesc, dict(CONV, num_tokens=4) if "step" in name else CONV, kw)
        refused(rp, name, d, fake(rp.RssmConvTables, y=0x20000), status, "" if "step" in name and "num_" in text else text)


@pytest.mark.parametrize("kw,status,text", BAD_SCAN)
def test_scan_scalars(rp, kw, status, text):
    d, n = build(rp.RssmScanDesc, SCAN, kw), ctypes.c_int64()
    refused(rp, "rssm_selective_scan", d, fake(rp.RssmScanTables), status, text)
    assert rp.lib().rssm_selective_scan_workspace(ctypes.byref(d), ctypes.byref(n)) == status


@pytest.mark.parametrize("kw,status,text", BAD_ROT)
def test_rotary_scalars(rp, kw, status, text):
    refused(rp, "rssm_rotary_append", build(rp.RssmRotaryDesc, ROT, kw), fake(rp.RssmRotaryTables), status, text)


@pytest.mark.parametrize("name,kw,status,text", [(n, *c) for n, cs in POOL_CALLS.items() for c in cs])
def test_pool_scalars(rp, name, kw, status, text):
    refused(rp, name, build(rp.RssmPagesDesc, PAGES, kw), fake(rp.RssmPagesTables), status, text)


def tables(rp, name, desc, cls, need, align16, align4, **base):
    lib = getattr(rp.lib(), name)
    assert lib(None, ctypes.byref(fake(cls, **base)), None) == 1
    assert lib(ctypes.byref(desc), None, None) == 1
    for f in need:
        refused(rp, name, desc, fake(cls, **{**base, f: None}), 1, f)
    for f in align16:
        refused(rp, name, desc, fake(cls, **{**base, f: 0x30008}), 1, "16-byte")
    for f in align4:
        refused(rp, name, desc, fake(cls, **{**base, f: 0x30002}), 1, "4-byte")


def test_conv_tables(rp):
    d = build(rp.RssmConvDesc, CONV, {})
    tables(rp, "rssm_causal_conv", d, rp.RssmConvTables, ("x", "weight", "y", "state", "slots", "seq_start"),
           ("x", "weight", "bias", "y", "state"), ("slots", "seq_start", "load_state"), y=0x20000)
    refused(rp, "rssm_causal_conv", d, fake(rp.RssmConvTables), 1, "y may not be x")
    refused(rp, "rssm_causal_conv_step", d, fake(rp.RssmConvTables), 1, "one row per request")
    for name in ("rssm_causal_conv", "rssm_causal_conv_step"):
        e = build(rp.RssmConvDesc, CONV, dict(num_seqs=0, num_tokens=0))
        assert getattr(rp.lib(), name)(ctypes.byref(e), ctypes.byref(fake(rp.RssmConvTables)), None) == 0
    big = build(rp.RssmConvDesc, CONV, dict(num_seqs=2 ** 27, num_tokens=2 ** 27))
    refused(rp, "rssm_causal_conv", big, fake(rp.RssmConvTables, y=0x20000), 1, "2^24")
    refused(rp, "rssm_causal_conv_step", build(rp.RssmConvDesc, CONV, dict(num_seqs=2 ** 28, num_tokens=2 ** 28)),
            fake(rp.RssmConvTables), 1, "2^24")


def test_scan_tables(rp):
    d = build(rp.RssmScanDesc, SCAN, {})
    tables(rp, "rssm_selective_scan", d, rp.RssmScanTables, ("state", "A", "x", "dt", "B", "C", "y", "slots", "seq_start"),
           ("state", "A", "D", "dt_bias", "x", "dt", "B", "C", "z", "y", "workspace"), ("slots", "seq_start", "load_state"))
    refused(rp, "rssm_selective_scan_step", d, fake(rp.RssmScanTables), 1, "one row per request")
    assert rp.lib().rssm_selective_scan_workspace(ctypes.byref(d), None) == 1
    for name in ("rssm_selective_scan", "rssm_selective_scan_step"):
        e = build(rp.RssmScanDesc, SCAN, dict(num_seqs=0, num_tokens=0))
        assert getattr(rp.lib(), name)(ctypes.byref(e), ctypes.byref(fake(rp.RssmScanTables)), None) == 0
        big = build(rp.RssmScanDesc, SCAN, dict(num_seqs=2 ** 26, num_tokens=2 ** 26))
        refused(rp, name, big, fake(rp.RssmScanTables), 1, "2^24")


def test_scan_workspace(rp):
    lib, n = rp.lib(), ctypes.c_int64()
    full = build(rp.RssmScanDesc, SCAN, dict(num_seqs=200, max_seq_len=5000))
    assert lib.rssm_selective_scan_workspace(ctypes.byref(full), ctypes.byref(n)) == 0 and n.value == 0
    few = build(rp.RssmScanDesc, SCAN, dict(num_seqs=1, max_seq_len=5000))
    assert lib.rssm_selective_scan_workspace(ctypes.byref(few), ctypes.byref(n)) == 0 and n.value > 0
    assert n.value % (1024 * 17 * 4) == 0          # [stretch][channel] of 16 states and a sum
    for ws, size in ((None, n.value), (0x10000, n.value - 1)):
        few.workspace_bytes = size
        refused(rp, "rssm_selective_scan", few, fake(rp.RssmScanTables, workspace=ws), 1, "workspace")


def test_rotary_tables(rp):
    d = build(rp.RssmRotaryDesc, ROT, {})
    tables(rp, "rssm_rotary_append", d, rp.RssmRotaryTables,
           ("q", "q_out", "k_new", "v_new", "k_cache", "v_cache", "page_table", "seq_start", "kv_len", "inv_freq"),
           ("q", "q_out", "k_new", "v_new", "k_cache", "v_cache"), ("page_table", "seq_start", "kv_len", "positions", "inv_freq"))
    alone = build(rp.RssmRotaryDesc, ROT, dict(num_kv_heads=0))
    refused(rp, "rssm_rotary_append", alone, fake(rp.RssmRotaryTables, positions=None, kv_len=None), 1, "kv_len")
    for kw in (dict(num_tokens=0), dict(num_q_heads=0, num_kv_heads=0), dict(num_seqs=0)):
        assert rp.lib().rssm_rotary_append(ctypes.byref(build(rp.RssmRotaryDesc, ROT, kw)), ctypes.byref(fake(rp.RssmRotaryTables)), None) == 0


def test_pool_tables(rp):
    d = build(rp.RssmPagesDesc, PAGES, {})
    rows = ("page_table", "kv_len", "page_ref")
    tables(rp, "rssm_page_extend", d, rp.RssmPagesTables, rows + ("dst", "lengths", "status", "workspace"), ("workspace",),
           rows + ("dst", "lengths", "status"))
    tables(rp, "rssm_page_fork", d, rp.RssmPagesTables, rows + ("src", "dst", "status", "cache_ptrs", "workspace"), ("workspace",),
           rows + ("src", "dst", "lengths", "status"))
    tables(rp, "rssm_page_release", d, rp.RssmPagesTables, rows + ("dst",), (), rows + ("dst", "lengths"))
    tables(rp, "rssm_page_compact", d, rp.RssmPagesTables, rows + ("live", "cache_ptrs", "workspace"), ("workspace",), rows + ("live",))
    tables(rp, "rssm_page_copy", d, rp.RssmPagesTables, ("src", "dst", "cache_ptrs"), (), ("src", "dst"))
    for name in ("rssm_page_extend", "rssm_page_fork", "rssm_page_release", "rssm_page_copy"):
        e = build(rp.RssmPagesDesc, PAGES, dict(num_items=0))
        assert getattr(rp.lib(), name)(ctypes.byref(e), ctypes.byref(fake(rp.RssmPagesTables)), None) == 0
        if name != "rssm_page_release" and name != "rssm_page_extend":
            big = build(rp.RssmPagesDesc, PAGES, dict(num_items=2 ** 20, num_caches=65535, workspace_bytes=1 << 40))
            refused(rp, name, big, fake(rp.RssmPagesTables), 1, "2^31")
    big = build(rp.RssmPagesDesc, PAGES, dict(num_pages=2 ** 30, num_caches=65535, workspace_bytes=1 << 40))
    refused(rp, "rssm_page_compact", big, fake(rp.RssmPagesTables), 1, "2^31")
    for name in ("rssm_page_fork", "rssm_page_compact", "rssm_page_copy"):
        refused(rp, name, d, fake(rp.RssmPagesTables, cache_ptrs=0x10004), 1, "8-byte")


def test_pool_workspace(rp):
    need = rp.rssm_pages_workspace(num_items=3, num_rows=8, num_pages=100)
    assert need >= 4 * (8 + 3 * 3 + 2 * 100 + 2)
    for name in ("rssm_page_extend", "rssm_page_fork"):
        for ws, size in ((None, need), (0x10000, need - 1)):
            refused(rp, name, build(rp.RssmPagesDesc, PAGES, dict(workspace_bytes=size)), fake(rp.RssmPagesTables, workspace=ws), 1, "workspace")
    small = rp.rssm_pages_workspace(num_items=0, num_rows=8, num_pages=100)
    refused(rp, "rssm_page_compact", build(rp.RssmPagesDesc, PAGES, dict(workspace_bytes=small - 1)), fake(rp.RssmPagesTables), 1, "workspace")
    with pytest.raises(rp.RssmError, match="num_rows"):
        rp.rssm_pages_workspace(num_items=1, num_rows=0, num_pages=1)


def test_descriptors_match_the_headers(rp):
    root = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    for header, pairs in (("rssm_causal_conv.h", (("rssm_causal_conv_desc", rp.RssmConvDesc), ("rssm_causal_conv_tables", rp.RssmConvTables))),
                          ("rssm_selective_scan.h", (("rssm_selective_scan_desc", rp.RssmScanDesc), ("rssm_selective_scan_tables", rp.RssmScanTables))),
                          ("rssm_rotary.h", (("rssm_rotary_desc", rp.RssmRotaryDesc), ("rssm_rotary_tables", rp.RssmRotaryTables))),
                          ("rssm_pages.h", (("rssm_pages_desc", rp.RssmPagesDesc), ("rssm_pages_tables", rp.RssmPagesTables)))):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, header)).read(), flags=re.S)
        for name, cls in pairs:
            body = next(b for b, n in re.findall(r"typedef struct \{(.*?)\} (\w+);", text, flags=re.S) if n == name)
            size = {"int32_t": 4, "float": 4, "int64_t": 8}
            want = [(m[2], 8 if m[1] else size[m[0]]) for m in re.findall(r"(?:const )?(\w+) ?(\*?)(\w+);", body)]
            assert [(n, ctypes.sizeof(t)) for n, t in cls._fields_] == want


def test_binding_refuses_host_tensors(rp):
    z = torch.zeros
    i = lambda *s: z(*s, dtype=torch.int32)                      # noqa: E731
    with pytest.raises(ValueError, match="device tensor"):
        rp.rssm_causal_conv(z(3, 8), z(4, 8), z(3, 8), z(2, 3, 8), i(1), i(2), stream=0)
    with pytest.raises(ValueError, match="device tensor"):
        rp.rssm_selective_scan_step(z(2, 8, 16), z(8, 16), z(1, 8), z(1, 1, 16), z(1, 1, 16), z(1, 8), z(1, 8), i(1), stream=0)
    with pytest.raises(ValueError, match="device tensor"):
        rp.rssm_rotary_append(z(1, 2, 64), z(1, 2, 64), None, None, None, None, None, None, None, z(32), positions=i(1), stream=0)
    with pytest.raises(ValueError, match="device tensor"):
        rp.rssm_page_release(i(2, 3), i(2), i(5), i(1), page_size=16, stream=0)
    with pytest.raises(ValueError, match="come together"):
        rp.rssm_rotary_append(None, z(1, 2, 64), None, None, None, None, None, None, None, z(32), stream=0)
    with pytest.raises(ValueError, match="comes with"):
        rp.rssm_rotary_append(None, None, None, None, z(1, 2, 64), None, None, None, None, z(32), stream=0)
    with pytest.raises(ValueError, match="come with"):
        rp.rssm_rotary_append(None, None, z(1, 16, 2, 64), None, None, None, None, None, None, z(32), stream=0)


def test_frequencies(rp):
    f, factor = rp.rotary_frequencies(64, 10000.0)
    assert factor == 1.0 and f.dtype == torch.float32 and f.shape == (32,)
    want = torch.tensor([10000.0 ** (-i / 32) for i in range(32)], dtype=torch.float64)
    assert ((f.double() - want).abs() <= 2.0 ** -23 * want).all()
    lin, _ = rp.rotary_frequencies(64, scale=4.0)
    assert ((lin.double() - want / 4).abs() <= 2.0 ** -23 * want).all()
    b, _ = rp.rotary_frequencies(64, scale=4.0, kind="base")
    assert b[0] == 1 and abs(float(b[-1]) * 4 / float(want[-1]) - 1) <= 2.0 ** -22
    m, factor = rp.rotary_frequencies(64, scale=4.0, kind="blend", trained=4096)
    turns = 4096 * want / (2 * math.pi)
    assert abs(factor - (0.1 * math.log(4.0) + 1)) < 1e-12
    assert torch.equal(m[turns >= 32], f[turns >= 32])
    slow = turns <= 1
    assert slow.any() and ((m.double() - want / 4).abs() <= 2.0 ** -23 * want)[slow].all()
    assert (m <= f).all() and (m.double() >= want / 4 * (1 - 2.0 ** -22)).all()
    assert rp.rotary_frequencies(16, kind="blend", trained=100, scale=0.5)[1] == 1.0
    for kw in (dict(kind="other"), dict(kind="blend"), dict(scale=0.0), dict(base=-1.0), dict(scale=math.inf)):
        with pytest.raises(ValueError):
            rp.rotary_frequencies(64, **kw)
    with pytest.raises(ValueError):
        rp.rotary_frequencies(63)


def test_host_pool_model():
    """The model that the GPU tests compare with, on a case worked out by hand."""
    from more_operators_ref import Pool
    p = Pool([[-1] * 3 for _ in range(4)], [0] * 4, [0] * 6, 4)
    assert p.extend([1, 0], [5, 4]) == [0, 0] and p.table[1][:2] == [0, 1] and p.table[0][0] == 2
    assert p.fork([1], [2], [None]) == [0] and p.table[2][:2] == [0, 3] and p.ref == [2, 1, 1, 1, 0, 0] and p.copies == [(1, 3, 1)]
    p.release([1])
    assert p.ref == [1, 0, 1, 1, 0, 0] and p.compact() == 3 and p.table[2][:2] == [0, 1] and p.ref == [1, 1, 1, 0, 0, 0]
    assert p.extend([3, 0], [12, 1]) == [0, 1]
