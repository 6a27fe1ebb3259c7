"""Host-side refusals of the prompt-side operators: bad arguments return before
any HIP call, so nothing here needs a GPU or launches a kernel."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def rp():
    import replayssm_persistent_rssm_amd as rp
    return rp


def fake(cls, **override):
    """Aligned, non-NULL addresses that are never dereferenced."""
    t = cls(**{f: 0x10000 for f, _ in cls._fields_})
    for k, v in override.items():
        setattr(t, k, v)
    return t


def lin_desc(rp, **kw):
    H, G = 64, 8
    base = dict(num_seqs=4, num_tokens=100, num_heads=H, heads_per_group=8, dim=64, dstate=128, num_slots=8,
                pad_slot_id=-1, max_seq_len=40, state_dtype=0, input_dtype=1, dt_softplus=1,
                state_slot_stride=H * 64 * 128, x_token_stride=H * 64, B_token_stride=G * 128, C_token_stride=G * 128,
                dt_token_stride=H, z_token_stride=H * 64, y_token_stride=H * 64, workspace_bytes=0)
    base.update(kw)
    return rp.RssmLinearDesc(**base)


BAD_LINEAR = [
    (dict(num_seqs=-1), 1, "num_seqs"), (dict(num_tokens=-1), 1, "num_tokens"), (dict(num_heads=0), 1, "num_heads"),
    (dict(heads_per_group=7), 1, "divide"), (dict(num_slots=0), 1, "num_slots"), (dict(max_seq_len=-1), 1, "max_seq_len"), (dict(max_seq_len=2 ** 30 + 1), 1, "max_seq_len"),
    (dict(dt_softplus=2), 1, "dt_softplus"), (dict(state_dtype=9), 1, "dtype"), (dict(state_dtype=3), 2, "f32, bf16 or f16"),
    (dict(input_dtype=4), 2, "f32, bf16 or f16"), (dict(dim=32), 2, "dim=32"), (dict(dstate=256), 2, "dstate=256"),
    (dict(state_slot_stride=100), 1, "state_slot_stride"), (dict(state_slot_stride=64 * 64 * 128 + 2), 1, "16 bytes"),
    (dict(x_token_stride=64 * 64 - 8), 1, "x_token_stride"), (dict(B_token_stride=8 * 128 + 4), 1, "B_token_stride"),
    (dict(C_token_stride=2 ** 23), 1, "C_token_stride"), (dict(dt_token_stride=63), 1, "dt_token_stride"),
    (dict(y_token_stride=1), 1, "y_token_stride"), (dict(z_token_stride=0), 1, "z_token_stride"),
    (dict(workspace_bytes=-1), 1, "workspace_bytes"), (dict(num_slots=2 ** 31 - 1, state_slot_stride=2 ** 44), 1, "2^46"),
]


@pytest.mark.parametrize("kw,status,text", BAD_LINEAR)
def test_linear_attention_scalars(rp, kw, status, text):
    d, t, n = lin_desc(rp, **kw), fake(rp.RssmLinearTables), ctypes.c_int64()
    assert rp.lib().rssm_linear_attention(ctypes.byref(d), ctypes.byref(t), None) == status
    assert text in rp.rssm_last_error()
    assert rp.lib().rssm_linear_attention_workspace(ctypes.byref(d), ctypes.byref(n)) == status


def test_linear_attention_tables(rp):
    lib, d = rp.lib(), lin_desc(rp)
    assert lib.rssm_linear_attention(None, ctypes.byref(fake(rp.RssmLinearTables)), None) == 1
    assert lib.rssm_linear_attention(ctypes.byref(d), None, None) == 1
    assert lib.rssm_linear_attention_workspace(ctypes.byref(d), None) == 1
    for f in ("state", "A", "x", "B", "C", "y", "slots", "seq_start"):
        assert lib.rssm_linear_attention(ctypes.byref(d), ctypes.byref(fake(rp.RssmLinearTables, **{f: None})), None) == 1
        assert f in rp.rssm_last_error()
    for f in ("state", "x", "B", "C", "z", "y", "workspace"):
        assert lib.rssm_linear_attention(ctypes.byref(d), ctypes.byref(fake(rp.RssmLinearTables, **{f: 0x10008})), None) == 1
        assert "16-byte" in rp.rssm_last_error()
    for f in ("A", "D", "dt_bias", "dt", "slots", "seq_start", "load_state"):
        assert lib.rssm_linear_attention(ctypes.byref(d), ctypes.byref(fake(rp.RssmLinearTables, **{f: 0x10002})), None) == 1
        assert "4-byte" in rp.rssm_last_error()
    # no dt: neither bias nor softplus
    for kw, tab in ((dict(dt_softplus=1), dict(dt=None, dt_bias=None)), (dict(dt_softplus=0), dict(dt=None))):
        assert lib.rssm_linear_attention(ctypes.byref(lin_desc(rp, **kw)), ctypes.byref(fake(rp.RssmLinearTables, **tab)), None) == 1
        assert "without dt" in rp.rssm_last_error()
    # nothing to enqueue
    assert lib.rssm_linear_attention(ctypes.byref(lin_desc(rp, num_seqs=0)), ctypes.byref(fake(rp.RssmLinearTables)), None) == 0


def test_linear_attention_workspace(rp):
    lib, n = rp.lib(), ctypes.c_int64()
    full = lin_desc(rp, num_seqs=8, max_seq_len=5000, num_tokens=40000)      # 512 (sequence, head) tiles
    assert lib.rssm_linear_attention_workspace(ctypes.byref(full), ctypes.byref(n)) == 0 and n.value == 0
    few = lin_desc(rp, num_seqs=1, max_seq_len=5000, num_tokens=5000)
    assert lib.rssm_linear_attention_workspace(ctypes.byref(few), ctypes.byref(n)) == 0 and n.value > 0
    for ws, size in ((None, n.value), (0x10000, n.value - 1)):
        few.workspace_bytes = size
        assert lib.rssm_linear_attention(ctypes.byref(few), ctypes.byref(fake(rp.RssmLinearTables, workspace=ws)), None) == 1
        assert "workspace" in rp.rssm_last_error()


def test_linear_attention_step(rp):
    lib = rp.lib()
    d = lin_desc(rp, num_seqs=4, num_tokens=5)
    assert lib.rssm_linear_attention_step(ctypes.byref(d), ctypes.byref(fake(rp.RssmLinearTables)), None) == 1
    assert "one row per request" in rp.rssm_last_error()
    d = lin_desc(rp, num_seqs=4, num_tokens=4)
    assert lib.rssm_linear_attention_step(ctypes.byref(d), None, None) == 1
    assert lib.rssm_linear_attention_step(ctypes.byref(d), ctypes.byref(fake(rp.RssmLinearTables, y=None)), None) == 1
    assert lib.rssm_linear_attention_step(ctypes.byref(lin_desc(rp, num_seqs=0, num_tokens=0)),
                                          ctypes.byref(fake(rp.RssmLinearTables)), None) == 0


def paged_desc(rp, **kw):
    base = dict(num_seqs=2, num_tokens=10, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_pages=100,
                max_pages=50, max_seq_len=8, max_kv_len=700, window=0, sinks=0, dtype=1, scale=0.1,
                page_stride=16 * 256, row_stride=256, head_stride=128, q_token_stride=1024, out_token_stride=1024,
                new_token_stride=256, table_stride=50, workspace_bytes=0)
    base.update(kw)
    return rp.RssmPagedDesc(**base)


BOTH = [
    (dict(num_seqs=-1), 1, "num_seqs"), (dict(num_tokens=-2), 1, "num_tokens"), (dict(num_kv_heads=0), 1, "num_kv_heads"),
    (dict(page_size=0), 1, "page_size"), (dict(num_pages=0), 1, "num_pages"), (dict(max_pages=0), 1, "max_pages"),
    (dict(dtype=7), 1, "dtype"), (dict(dtype=3), 2, "f32, bf16 or f16"), (dict(head_dim=96), 2, "head_dim=96"),
    (dict(page_stride=64), 1, "page_stride"), (dict(row_stride=260), 1, "row_stride"), (dict(head_stride=0), 1, "head_stride"),
    (dict(table_stride=49), 1, "table_stride"),
]
ATTEND = [
    (dict(num_q_heads=7), 1, "divide"), (dict(max_seq_len=-1), 1, "max_seq_len"), (dict(max_kv_len=2 ** 30 + 1), 1, "max_kv_len"),
    (dict(window=-1), 1, "window"), (dict(sinks=-1), 1, "sinks"), (dict(scale=0.0), 1, "scale"),
    (dict(scale=float("nan")), 1, "scale"), (dict(scale=float("inf")), 1, "scale"),
    (dict(q_token_stride=1020), 1, "q_token_stride"), (dict(out_token_stride=1028), 1, "out_token_stride"),
    (dict(workspace_bytes=-1), 1, "workspace_bytes"), (dict(max_seq_len=2 ** 24, num_q_heads=512), 1, "2^30"),
]


@pytest.mark.parametrize("kw,status,text", BOTH + ATTEND)
def test_paged_attention_scalars(rp, kw, status, text):
    d, t, n = paged_desc(rp, **kw), fake(rp.RssmPagedTables), ctypes.c_int64()
    assert rp.lib().rssm_paged_attention(ctypes.byref(d), ctypes.byref(t), None) == status
    assert text in rp.rssm_last_error()
    assert rp.lib().rssm_paged_attention_workspace(ctypes.byref(d), ctypes.byref(n)) == status


@pytest.mark.parametrize("kw,status,text", BOTH + [(dict(new_token_stride=255), 1, "new_token_stride")])
def test_paged_append_scalars(rp, kw, status, text):
    d, t = paged_desc(rp, **kw), fake(rp.RssmPagedTables)
    assert rp.lib().rssm_paged_append(ctypes.byref(d), ctypes.byref(t), None) == status
    assert text in rp.rssm_last_error()


def test_paged_tables(rp):
    lib, d = rp.lib(), paged_desc(rp)
    for fn, need in ((lib.rssm_paged_attention, ("k_cache", "v_cache", "q", "out", "page_table", "seq_start", "kv_len")),
                     (lib.rssm_paged_append, ("k_cache", "v_cache", "k_new", "v_new", "page_table", "seq_start", "kv_len"))):
        assert fn(None, ctypes.byref(fake(rp.RssmPagedTables)), None) == 1
        assert fn(ctypes.byref(d), None, None) == 1
        for f in need:
            assert fn(ctypes.byref(d), ctypes.byref(fake(rp.RssmPagedTables, **{f: None})), None) == 1
            assert f in rp.rssm_last_error()
            assert fn(ctypes.byref(d), ctypes.byref(fake(rp.RssmPagedTables, **{f: 0x10002})), None) == 1
            assert "aligned" in rp.rssm_last_error()
        for kw in (dict(num_seqs=0), dict(num_tokens=0)):
            assert fn(ctypes.byref(paged_desc(rp, **kw)), ctypes.byref(fake(rp.RssmPagedTables)), None) == 0
    assert lib.rssm_paged_attention(ctypes.byref(d), ctypes.byref(fake(rp.RssmPagedTables, lse=0x10002)), None) == 1
    assert lib.rssm_paged_attention_workspace(ctypes.byref(d), None) == 1


def test_paged_workspace(rp):
    lib, n = rp.lib(), ctypes.c_int64()
    d = paged_desc(rp, num_seqs=1, max_seq_len=1, num_tokens=1, max_kv_len=100000)
    assert lib.rssm_paged_attention_workspace(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    assert n.value % (8 * 130 * 4) == 0            # [head][split] of 128 outputs, a maximum and a sum
    for ws, size in ((None, n.value), (0x10000, n.value - 1)):
        d.workspace_bytes = size
        assert lib.rssm_paged_attention(ctypes.byref(d), ctypes.byref(fake(rp.RssmPagedTables, workspace=ws)), None) == 1
        assert "workspace" in rp.rssm_last_error()
    d = paged_desc(rp, num_seqs=1, max_seq_len=1, num_tokens=1, max_kv_len=100)
    assert lib.rssm_paged_attention_workspace(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value == 0
    # a window bounds the tiles however long the cache is
    d = paged_desc(rp, num_seqs=1, max_seq_len=1, num_tokens=1, max_kv_len=2 ** 30, window=64)
    assert lib.rssm_paged_attention_workspace(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value == 0


def norm_desc(rp, **kw):
    base = dict(rows=4, channels=1024, groups=8, input_dtype=1, residual_dtype=0, eps=1e-5, residual_scale=1.0,
                y_row_stride=1024, z_row_stride=1024, residual_row_stride=1024, residual_out_row_stride=1024,
                normed_row_stride=1024)
    base.update(kw)
    return rp.RssmNormDesc(**base)


BAD_NORM = [
    (dict(rows=-1), 1, "rows"), (dict(channels=0), 1, "channels"), (dict(channels=1020), 1, "channels"),
    (dict(channels=16392), 1, "channels"), (dict(groups=0), 1, "groups"), (dict(groups=3), 1, "groups"),
    (dict(groups=256), 1, "groups"), (dict(channels=16384, groups=512), 1, "groups"), (dict(input_dtype=8), 1, "dtype"),
    (dict(input_dtype=3), 2, "f32, bf16 or f16"), (dict(residual_dtype=4), 2, "f32, bf16 or f16"),
    (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"), (dict(y_row_stride=1000), 1, "y_row_stride"),
    (dict(z_row_stride=1028), 1, "z_row_stride"), (dict(residual_row_stride=1026), 1, "residual_row_stride"),
    (dict(residual_out_row_stride=8), 1, "residual_out_row_stride"), (dict(normed_row_stride=2 ** 32), 1, "normed_row_stride"),
]


@pytest.mark.parametrize("kw,status,text", BAD_NORM)
def test_block_norm_scalars(rp, kw, status, text):
    d, t = norm_desc(rp, **kw), fake(rp.RssmNormTables)
    assert rp.lib().rssm_block_norm(ctypes.byref(d), ctypes.byref(t), None) == status
    assert text in rp.rssm_last_error()


def test_block_norm_tables(rp):
    lib, d = rp.lib(), norm_desc(rp)
    assert lib.rssm_block_norm(None, ctypes.byref(fake(rp.RssmNormTables)), None) == 1
    assert lib.rssm_block_norm(ctypes.byref(d), None, None) == 1
    for f in ("y", "residual", "residual_out"):
        assert lib.rssm_block_norm(ctypes.byref(d), ctypes.byref(fake(rp.RssmNormTables, **{f: None})), None) == 1
        assert f in rp.rssm_last_error()
    for f, _ in rp.RssmNormTables._fields_:
        assert lib.rssm_block_norm(ctypes.byref(d), ctypes.byref(fake(rp.RssmNormTables, **{f: 0x10008})), None) == 1
        assert "16-byte" in rp.rssm_last_error()
    assert lib.rssm_block_norm(ctypes.byref(d), ctypes.byref(fake(rp.RssmNormTables, normed=None)), None) == 1
    assert "pre_weight" in rp.rssm_last_error()
    assert lib.rssm_block_norm(ctypes.byref(norm_desc(rp, rows=0)), ctypes.byref(fake(rp.RssmNormTables)), None) == 0


def test_binding_refuses_host_tensors(rp):
    """The binding names the first tensor that is not on a device."""
    z = torch.zeros
    i = lambda *s: z(*s, dtype=torch.int32)                      # noqa: E731
    with pytest.raises(ValueError, match="device tensor"):
        rp.rssm_linear_attention(z(2, 4, 64, 128), z(4), z(3, 4, 64), z(3, 2, 128), z(3, 2, 128), z(3, 4), z(3, 4, 64), i(1),
                                 i(2), max_seq_len=3, stream=0)
    with pytest.raises(ValueError, match="device tensor"):
        rp.rssm_paged_append(z(4, 16, 2, 64), z(4, 16, 2, 64), z(1, 2, 64), z(1, 2, 64), i(1, 4), i(2), i(1), stream=0)
    with pytest.raises(ValueError, match="device tensor"):
        rp.rssm_block_norm(z(2, 64), z(2, 64), z(2, 64), stream=0)
    with pytest.raises(TypeError):
        rp.rssm_linear_attention_step(None, z(4), z(3, 4, 64), z(3, 2, 128), z(3, 2, 128), z(3, 4), z(3, 4, 64), i(3), stream=0)
    with pytest.raises(TypeError):
        rp.rssm_linear_attention_step(z(2, 4, 64, 128), z(4), z(3, 4, 64), z(3, 2, 128), z(3, 2, 128), z(3, 4), z(3, 4, 64),
                                      i(3), load_state=i(3))


def test_descriptors_match_the_headers(rp):
    """Field order of the binding's structures against the C declarations."""
    import os
    import re
    root = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    for header, pairs in (("rssm_linear_attention.h", (("rssm_linear_attention_desc", rp.RssmLinearDesc),
                                                       ("rssm_linear_attention_tables", rp.RssmLinearTables))),
                          ("rssm_paged_attention.h", (("rssm_paged_attention_desc", rp.RssmPagedDesc),
                                                      ("rssm_paged_attention_tables", rp.RssmPagedTables))),
                          ("rssm_block_norm.h", (("rssm_block_norm_desc", rp.RssmNormDesc),
                                                 ("rssm_block_norm_tables", rp.RssmNormTables)))):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, header)).read(), flags=re.S)
        for name, cls in pairs:
            body = next(b for b, n in re.findall(r"typedef struct \{(.*?)\} (\w+);", text, flags=re.S) if n == name)
            size = {"int32_t": 4, "float": 4, "int64_t": 8}
            want = [(m[2], 8 if m[1] else size[m[0]]) for m in
                    re.findall(r"(?:const )?(\w+) ?(\*?)(\w+);", body)]
            assert [(n, ctypes.sizeof(t)) for n, t in cls._fields_] == want


def test_more_workgroups_than_one_launch_takes(rp):
    """Refused by name before any HIP call."""
    lib = rp.lib()
    for fn, kw in ((lib.rssm_linear_attention, dict(num_seqs=2 ** 18)),
                   (lib.rssm_linear_attention_step, dict(num_seqs=2 ** 18, num_tokens=2 ** 18))):
        assert fn(ctypes.byref(lin_desc(rp, **kw)), ctypes.byref(fake(rp.RssmLinearTables)), None) == 1
        assert "2^24" in rp.rssm_last_error()
    tab = fake(rp.RssmPagedTables)
    wide = dict(num_seqs=2 ** 16, max_seq_len=2 ** 14, num_tokens=2 ** 30)
    assert lib.rssm_paged_attention(ctypes.byref(paged_desc(rp, **wide)), ctypes.byref(tab), None) == 1
    assert "2^24" in rp.rssm_last_error()
    assert lib.rssm_paged_append(ctypes.byref(paged_desc(rp, num_tokens=2 ** 28)), ctypes.byref(tab), None) == 1
    assert "2^24" in rp.rssm_last_error()
