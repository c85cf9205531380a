"""C-ABI checks that need no GPU: the library loads, exports every symbol
include/tl.h declares, validates configurations, and sizes its weight blob and
workspace by formulas checked here independently."""
import ctypes as C
import os
import re

import pytest

import synthetic as S
import dynamic_depth_b200 as T
from dynamic_depth_b200 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def header_functions():
    src = open(os.path.join(ROOT, "include", "tl.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(tl_[a-z0-9_]+)\s*\(", src)))


def test_library_exports_every_declared_symbol():
    lib = _lib.lib()
    names = header_functions()
    assert len(names) >= 17
    for n in names:
        assert hasattr(lib, n), n
        assert n in _lib.SIGNATURES, n


def test_strerror_names_every_status():
    lib = _lib.lib()
    seen = set()
    for s in range(0, -8, -1):
        msg = lib.tl_strerror(s).decode()
        assert msg and msg != "unknown status"
        seen.add(msg)
    assert len(seen) == 8
    assert lib.tl_strerror(-99).decode() == "unknown status"


def _blob_formula(shape, group):
    """Bytes of the weight blob, counted from the shapes."""
    d, F, V = shape.d, shape.ffn, shape.vocab

    def mat(fmt, n, k):
        return n * k // 2 + n * (k // group) * 2 if fmt == "int4" else n * k * 2

    total = 8 + 48
    total += 2 * mat(shape.fmt_embed_head, V, d)
    for b in range(shape.n_pre + shape.n_loop_layers):
        f = shape.fmt_pre if b < shape.n_pre else shape.fmt_loop
        total += mat(f, 3 * d, d) + mat(f, d, d) + 2 * mat(f, F, d) + mat(f, d, F)
    total += (2 * (shape.n_pre + shape.n_loop_layers) + 1) * d * 4
    return total


@pytest.mark.parametrize("name", ["tiny", "m407", "m407_bf16loop", "m1b4"])
def test_weight_blob_size_formula(name):
    sh = S.SHAPES[name]
    cfg = T.config_from_shape(sh, max_lanes=4, max_seq=128, L_max=8)
    assert T.weights_bytes(cfg) == _blob_formula(sh, cfg.group)


def test_407m_int4_loop_block_bytes():
    # one loop iteration of the 407M-class model reads 8,650,752 bytes of INT4 weights + scales
    sh = S.M407
    d, F, g = sh.d, sh.ffn, sh.group
    per = sum(n * k // 2 + n * (k // g) * 2 for n, k in [(3 * d, d), (d, d), (F, d), (F, d), (d, F)])
    assert per == 8_650_752


def test_workspace_grows_with_capacity_and_kv_formula():
    sh = S.M407
    a = T.workspace_bytes(T.config_from_shape(sh, max_lanes=1, max_seq=128, L_max=8))
    b = T.workspace_bytes(T.config_from_shape(sh, max_lanes=2, max_seq=128, L_max=8))
    # one more lane adds at least its KV: (n_pre + L_max) slots x 2 pages x page bytes
    page = 2 * sh.n_heads * 64 * sh.head_dim * 2
    assert b - a >= (sh.n_pre + 8) * 2 * page
    c = T.workspace_bytes(T.config_from_shape(sh, max_lanes=1, max_seq=128, L_max=8, kv_pool_pages=10))
    assert a - c >= ((sh.n_pre + 8) * 2 - 10) * page


@pytest.mark.parametrize("field,value", [("d", 100), ("n_heads", 3), ("group", 48), ("kv_page_tokens", 48),
                                         ("ffn", 544),  # a multiple of 32 but not of 64
                                         ("ffn", 2048),  # 64 scale groups of 32 across ffn
                                         ("kv_page_tokens", 16), ("max_lanes", 0), ("max_lanes", 2048),
                                         ("L_max", 0), ("fmt_loop", 7), ("max_prefill_tokens", -1),
                                         ("act_split", 3), ("act_split", -1)])
def test_invalid_configs_rejected(field, value):
    cfg = T.config_from_shape(S.TINY, max_lanes=2, max_seq=64, L_max=4)
    setattr(cfg, field, value)
    n = C.c_size_t()
    assert _lib.lib().tl_workspace_bytes(C.byref(cfg), C.byref(n)) == _lib.TL_EINVAL
    assert _lib.lib().tl_weights_bytes(C.byref(cfg), C.byref(n)) == _lib.TL_EINVAL


def test_null_arguments_rejected_without_cuda():
    lib = _lib.lib()
    cfg = T.config_from_shape(S.TINY, max_lanes=2, max_seq=64, L_max=4)
    h = C.c_void_p()
    assert lib.tl_create(C.byref(cfg), None, 1 << 20, None, C.byref(h)) == _lib.TL_EINVAL
    assert lib.tl_create(C.byref(cfg), 0x1001, 1 << 20, None, C.byref(h)) == _lib.TL_EINVAL  # unaligned
    assert lib.tl_load_weights(None, None, 0) == _lib.TL_EINVAL
    assert lib.tl_decode(None, None, 1, 1, None, None) == _lib.TL_EINVAL
    assert lib.tl_quantize_int4(None, 4, 64, 32, None, None, None) == _lib.TL_EINVAL
    assert lib.tl_quantize_int4(0x1000, 4, 48, 32, 0x1000, 0x1000, None) == _lib.TL_EINVAL
    assert lib.tl_set_early_exit(None, 0.1, 2, 2, 1) == _lib.TL_EINVAL


def test_blob_header_layout():
    from dynamic_depth_b200 import weights as Wt
    cfg = T.config_from_shape(S.TINY, max_lanes=2, max_seq=64, L_max=4)
    h = Wt.header(cfg)
    assert len(h) == 56 and h[:8] == b"TLWBLOB1"
    assert Wt.gain_order(cfg) == S.gain_names(S.TINY)
    assert len(Wt.matrix_formats(cfg)) == len(S.matrix_shapes(S.TINY))


def test_prompt_rows_may_exceed_one_sequence():
    # a batched prefill computes the prompts of several lanes at once
    cfg = T.config_from_shape(S.TINY, max_lanes=8, max_seq=64, L_max=4, max_prefill_tokens=512)
    small = T.config_from_shape(S.TINY, max_lanes=8, max_seq=64, L_max=4)
    assert T.workspace_bytes(cfg) > T.workspace_bytes(small)


def _ws(sh, **kw):
    return T.workspace_bytes(T.config_from_shape(sh, **kw))


def test_split_activations_double_the_fp16_activation_copies():
    # act_split = 1 stores every fp16 activation copy as [hi | lo] rows: three copies (norm output,
    # attention output: d wide; SwiGLU output: ffn wide) for the prompt rows and again for the boundary
    # stage's scratch (max_lanes rows), each twice as wide
    sh = S.M407
    cap = dict(max_lanes=4, max_seq=128, L_max=8, max_prefill_tokens=512)
    single = _ws(sh, act_split=2, **cap)
    split = _ws(sh, act_split=1, **cap)
    rows, lanes = 512, 4
    extra = (rows + lanes) * (2 * sh.d + sh.ffn) * 2
    assert extra <= split - single <= extra + 6 * 256  # up to one alignment pad per region


def test_split_activations_automatic_past_48_blocks():
    # automatic: split when n_pre + L_max * n_loop_layers > 48 (the 407M-class model at L_max = 32 crosses
    # 34 blocks, the 1.4B-class layout at L_max = 4 crosses 96)
    m407 = dict(max_lanes=2, max_seq=64, max_prefill_tokens=64)
    assert _ws(S.M407, L_max=32, act_split=0, **m407) == _ws(S.M407, L_max=32, act_split=2, **m407)
    assert _ws(S.M407, L_max=47, act_split=0, **m407) == _ws(S.M407, L_max=47, act_split=1, **m407)
    mini = dict(max_lanes=2, max_seq=64, max_prefill_tokens=64)
    assert _ws(S.M1B4_MINI, L_max=16, act_split=0, **mini) == _ws(S.M1B4_MINI, L_max=16, act_split=2, **mini)
    assert _ws(S.M1B4_MINI, L_max=17, act_split=0, **mini) == _ws(S.M1B4_MINI, L_max=17, act_split=1, **mini)


def test_workspace_holds_a_resident_fp16_copy_of_every_block():
    # every block's five matrices in fp16: (3d*d + d*d + 2*ffn*d + d*ffn) halves per block
    sh = S.M407
    cfg = T.config_from_shape(sh, max_lanes=1, max_seq=64, L_max=2)
    ws = T.workspace_bytes(cfg)
    weights = T.weights_bytes(cfg)
    copies = (sh.n_pre + sh.n_loop_layers) * (4 * sh.d * sh.d + 3 * sh.d * sh.ffn) * 2
    assert ws > weights + copies


# ------------------------------------------------------- serving operators --
A = 0x1000  # an aligned address that nothing reads: every call here is refused before anything is enqueued


def test_plan_batch_row_limits():
    def plan(n_rows, parents):
        return _lib.lib().tl_plan_batch(A, A, 2, 16, A, 4, A, 3, A, parents, n_rows, 0, A, A + 128, A, A + 64, A, A, None,
                                        None, None)
    assert plan((1 << 30) + 1, None) == _lib.TL_EINVAL
    assert plan((1 << 31) - 1, None) == _lib.TL_EINVAL
    assert plan((1 << 20) + 1, A) == _lib.TL_EINVAL


def _pool(**kw):
    f = dict(dev_pool=A, n_pages=4, dtype=_lib.TL_F16, n_kv_heads=2, head_dim=64, page_tokens=16)
    f.update(kw)
    return C.byref(_lib.TlKvPool(**f))


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 20) + 1),
                                dict(stride=9), dict(n_top=-1), dict(n_top=65), dict(n_top=11), dict(x=None),
                                dict(x=A + 2), dict(targets=None), dict(n_top=0), dict(targets=A + 1), dict(ids=A + 2)])
def test_token_logprobs_refusals(kw):
    a = dict(x=A, dtype=_lib.TL_F32, rows=3, vocab=10, stride=10, targets=A, n_top=2, ids=A)
    a.update(kw)
    st = _lib.lib().tl_token_logprobs(a["x"], a["dtype"], a["rows"], a["vocab"], a["stride"], a["targets"], a["n_top"],
                                      A, A, A, A, a["ids"], A, None)
    assert st == _lib.TL_EINVAL


def test_operators_with_nothing_to_do():
    lib = _lib.lib()
    assert lib.tl_token_logprobs(None, 0, 0, 10, 10, None, 0, None, None, None, None, None, None, None) == 0
    assert lib.tl_norm_rope_append(None, 0, 0, 384, 2, None, None, 1e-6, None, 8, None, None, _pool(), None, None,
                                   None) == 0
    assert lib.tl_tree_attention(None, 128, _pool(), None, 4, None, None, 0, 0, 2, 1, None, 0, 0.0, None, 1, 128, None,
                                 None, 0, None, None) == 0


@pytest.mark.parametrize("kw", [dict(R=0), dict(R=8193), dict(page=0), dict(page=24), dict(page=8192), dict(mp=0),
                                dict(n_free=-1), dict(n_rows=-1), dict(words=9), dict(words=-1), dict(words=0),
                                dict(masks=None), dict(cached=None), dict(head_out=A), dict(lens=A), dict(slots=A + 4),
                                dict(free=None), dict(table=A + 2)])
def test_plan_batch_refusals(kw):
    a = dict(R=2, page=16, mp=4, n_free=3, n_rows=5, words=1, masks=A, cached=A, head_out=A + 64, lens=A + 128, slots=A,
             free=A, table=A)
    a.update(kw)
    st = _lib.lib().tl_plan_batch(a["cached"], A, a["R"], a["page"], a["table"], a["mp"], a["free"], a["n_free"], A,
                                  None, a["n_rows"], a["words"], A, a["lens"], A, a["head_out"], a["slots"], A,
                                  a["masks"], None, None)
    assert st == _lib.TL_EINVAL


BAD_POOLS = [dict(dev_pool=None), dict(dev_pool=A + 8), dict(n_pages=0), dict(dtype=_lib.TL_F32), dict(n_kv_heads=0),
             dict(head_dim=96), dict(page_tokens=8), dict(page_tokens=48), dict(page_tokens=2048),
             dict(n_pages=1 << 26)]


@pytest.mark.parametrize("kw", [dict(pool=p) for p in BAD_POOLS] + [
    dict(dtype=4), dict(rows=-1), dict(stride=380), dict(stride=385), dict(heads=3), dict(heads=0), dict(gq=A),
    dict(eps=-1.0), dict(eps=float("nan")), dict(length=0), dict(x=A + 8), dict(x=None), dict(slots=A + 4), dict(q=A + 2)])
def test_norm_rope_append_refusals(kw):
    a = dict(pool={}, dtype=_lib.TL_F16, rows=2, stride=384, heads=2, gq=None, eps=1e-6, length=8, x=A, slots=A, q=A)
    a.update(kw)
    st = _lib.lib().tl_norm_rope_append(a["x"], a["dtype"], a["rows"], a["stride"], a["heads"], a["gq"], None, a["eps"],
                                        A, a["length"], A, a["slots"], _pool(**a["pool"]), a["q"], None, None)
    assert st == _lib.TL_EINVAL


@pytest.mark.parametrize("kw", [dict(pool=p) for p in BAD_POOLS] + [
    dict(qs=120), dict(qs=132), dict(heads=3), dict(heads=0), dict(R=-1), dict(rows=-1), dict(mp=0), dict(nodes=0),
    dict(masks=None), dict(words=0), dict(nodes=33), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(od=_lib.TL_BF16), dict(od=5), dict(os=120), dict(q=None), dict(q=A + 2),
    dict(ws=None), dict(ws=A + 128), dict(lse=A + 1)])
def test_tree_attention_refusals(kw):
    a = dict(pool={}, qs=128, heads=2, R=2, rows=3, mp=4, nodes=8, masks=A, words=1, scale=0.0, od=_lib.TL_F16, os=128,
             q=A, ws=A, lse=A)
    a.update(kw)
    st = _lib.lib().tl_tree_attention(a["q"], a["qs"], _pool(**a["pool"]), A, a["mp"], A, A, a["R"], a["rows"],
                                      a["heads"], a["nodes"], a["masks"], a["words"], a["scale"], A, a["od"], a["os"],
                                      a["lse"], a["ws"], 1 << 30, None, None)
    assert st == _lib.TL_EINVAL


@pytest.mark.parametrize("kw", [dict(R=(1 << 20) + 1), dict(words=(1 << 20) + 1), dict(nodes=(1 << 30) + 1, masks=None),
                                dict(nodes=(1 << 31) - 1, masks=None), dict(scale=2e38)])
def test_tree_attention_size_limits(kw):
    a = dict(R=2, nodes=8, masks=A, words=1, scale=0.0)
    a.update(kw)
    words = a["words"] if a["masks"] else 0
    st = _lib.lib().tl_tree_attention(A, 128, _pool(), A, 4, A, A, a["R"], 3, 2, a["nodes"], a["masks"], words,
                                      a["scale"], A, _lib.TL_F16, 128, A, A, 1 << 62, None, None)
    assert st == _lib.TL_EINVAL


def test_rope_table_refusals():
    lib = _lib.lib()
    for table, length, hd, base in ((None, 4, 64, 1e4), (A + 4, 4, 64, 1e4), (A, 0, 64, 1e4), (A, 4, 63, 1e4),
                                    (A, 4, 0, 1e4), (A, 4, 64, 0.0), (A, 4, 64, float("nan"))):
        assert lib.tl_rope_table(table, length, hd, base, None) == _lib.TL_EINVAL


def test_operator_wrappers_refuse_host_tensors_and_shapes():
    import torch
    with pytest.raises(ValueError):
        T.token_logprobs(torch.zeros(2, 3), None, n_top=1)
    with pytest.raises(ValueError):
        T.token_logprobs(torch.zeros(2, 3, 4))
    with pytest.raises(ValueError):
        T.token_logprobs(torch.zeros(2, 3, dtype=torch.float64))
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        T.plan_batch(z, z, torch.zeros(3, 4, dtype=torch.int32), z, z[:1], 16, 2)
    pool = torch.zeros(2, 2, 1, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        T.norm_rope_append(torch.zeros(2, 100), 1, pool, z.long(), z, torch.zeros(4, 32, 2))
    with pytest.raises(ValueError):
        T.tree_attention(torch.zeros(2, 1, 64), pool, torch.zeros(1, 4, dtype=torch.int32), z[:1], z, 1)
    with pytest.raises(ValueError, match="masks"):  # no words is not the same as no masks
        T.tree_attention(torch.zeros(2, 1, 64, dtype=torch.float16), pool, torch.zeros(1, 4, dtype=torch.int32), z[:1], z,
                         1, masks=torch.zeros(2, 0, dtype=torch.int32))
