"""What the serving operators accept and refuse before anything is enqueued, through the C ABI (no GPU is needed)."""
import ctypes as C

import pytest
import torch

import dynamic_depth_b200 as T
from dynamic_depth_b200 import _lib

A = 0x100000  # an aligned address that nothing reads


def pool(**kw):
    f = dict(dev_pool=A, n_pages=4, dtype=_lib.TL_F16, n_kv_heads=2, head_dim=64, page_tokens=16)
    f.update(kw)
    return C.byref(_lib.TlKvPool(**f))


@pytest.mark.parametrize("R,rows", [(2, 0), (0, 0)])
def test_tree_attention_of_no_rows_needs_no_masks(R, rows):
    """The masks of an empty batch are an empty tensor, which has no address."""
    st = _lib.lib().tl_tree_attention(None, 128, pool(), A, 4, A, A, R, rows, 2, 8, None, 1, 0.0, None, _lib.TL_F16, 128,
                                      None, A, 1 << 30, None, None)
    assert st == _lib.TL_OK


def test_masks_are_still_wanted_where_there_are_rows():
    assert _lib.lib().tl_tree_attention(A, 128, pool(), A, 4, A, A, 2, 3, 2, 8, None, 1, 0.0, A, _lib.TL_F16, 128, None,
                                        A, 1 << 30, None, None) == _lib.TL_EINVAL


# buffers of a plan of 5 requests and 7 rows, each at an address of its own, and their sizes in bytes
PLAN = dict(cached=20, fresh=20, table=80, free=12, free_head=4, parents=28, cu=24, lens=20, granted=20, head_out=4,
            slots=56, positions=28, masks=56, status=4)
OUTPUTS = ("table", "cu", "lens", "granted", "head_out", "slots", "positions", "masks", "status")


@pytest.mark.parametrize("out", OUTPUTS)
def test_plan_outputs_share_no_byte_with_another_buffer(out):
    def plan(at):
        return _lib.lib().tl_plan_batch(at["cached"], at["fresh"], 5, 16, at["table"], 4, at["free"], 3,
                                        at["free_head"], at["parents"], 7, 2, at["cu"], at["lens"], at["granted"],
                                        at["head_out"], at["slots"], at["positions"], at["masks"], at["status"], None)
    apart = {k: A + 4096 * i for i, k in enumerate(PLAN)}
    for other, size in PLAN.items():
        if other == out:
            continue
        first = apart[other]
        last = first + size - (8 if out == "slots" else 4)  # the last place of the other's that this one's can start in
        for at in {first, max(first, last // 8 * 8 if out == "slots" else last)}:
            assert plan(dict(apart, **{out: at})) == _lib.TL_EINVAL, (other, at - first)


def _calls():
    """One call of each operator with floating inputs: the call and the names of those inputs."""
    z = torch.zeros(2, dtype=torch.int32)
    h = dict(dtype=torch.float16)

    def make():
        return dict(logits=torch.zeros(2, 5), qkv=torch.zeros(2, 192, **h), pool=torch.zeros(2, 2, 1, 16, 64, **h),
                    rope=torch.zeros(4, 32, 2), q_gain=torch.ones(64), k_gain=torch.ones(64),
                    q=torch.zeros(2, 1, 64, **h), out=torch.zeros(2, 1, 64, **h))
    return make, [
        (lambda d: T.token_logprobs(d["logits"], n_top=1), ("logits",)),
        (lambda d: T.norm_rope_append(d["qkv"], 1, d["pool"], z.long(), z, d["rope"], q_gain=d["q_gain"],
                                      k_gain=d["k_gain"], q_out=d["out"]),
         ("qkv", "pool", "rope", "q_gain", "k_gain", "out")),
        (lambda d: T.tree_attention(d["q"], d["pool"], torch.zeros(1, 4, dtype=torch.int32), z[:1], z, 1, out=d["out"]),
         ("q", "pool", "out"))]


def test_tensors_that_want_a_gradient_are_refused():
    make, calls = _calls()
    for call, names in calls:
        for name in names:
            d = make()
            d[name].requires_grad_(True)
            with pytest.raises(ValueError, match="backward"):
                call(d)
            with torch.no_grad(), pytest.raises(ValueError, match="cuda|CUDA|device"):  # host tensors: refused as such
                call(d)


@pytest.mark.parametrize("out,stride,dtype,rows", [
    (A + 16, 128, _lib.TL_F16, 3),           # inside the first row
    (A + 256, 128, _lib.TL_F16, 3),          # the next row
    (A - 256, 128, _lib.TL_F16, 3),
    (A, 256, _lib.TL_F16, 3),                # the same place with another stride
    (A, 128, _lib.TL_F32, 3),                # and with another type
    (A + 256, 256, _lib.TL_F16, 2),
    (A, 128, _lib.TL_F32, 1),
    (A + 16, 128, _lib.TL_F16, 1)])
def test_attention_outputs_beside_the_queries_or_in_their_place(out, stride, dtype, rows):
    st = _lib.lib().tl_tree_attention(A, 128, pool(dev_pool=2 * A), 3 * A, 4, 3 * A, 3 * A, 2, rows, 2, 8, None, 0, 0.0, out,
                                      dtype, stride, None, 4 * A, 1 << 30, None, None)
    assert st == _lib.TL_EINVAL


@pytest.mark.parametrize("shift", [16, 240, 272, 512 - 16, -16, -240, 512 + 128])
def test_attention_outputs_between_the_queries_rows(shift):
    """Rows of 256 bytes every 512: an output shifted by 256 fits between them, one shifted by less or more does not."""
    st = _lib.lib().tl_tree_attention(A, 256, pool(dev_pool=2 * A), 3 * A, 4, 3 * A, 3 * A, 2, 5, 2, 8, None, 0, 0.0,
                                      A + shift, _lib.TL_F16, 256, None, 4 * A, 1 << 30, None, None)
    assert st == _lib.TL_EINVAL
