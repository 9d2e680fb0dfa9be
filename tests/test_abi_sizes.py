"""Sizes that the C interface's 32-bit integers do not hold are refused, not cut
(host only: tensors without memory)."""
import pytest
import torch

from invariant_verify_gb300 import abi as B

BIG = (1 << 32) + 8                                # cut to 32 bits: 8
SHAPE = 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    from invariant_verify_gb300 import build
    build.build()
    return B.lib()


def bf(*s):
    return torch.empty(*s, dtype=torch.bfloat16, device="meta")


def i32(*s):
    return torch.empty(*s, dtype=torch.int32, device="meta")


def f32(*s):
    return torch.empty(*s, device="meta")


def refused(fn, *args, **kw):
    with pytest.raises(B.BivError) as e:
        fn(*args, **kw)
    assert e.value.status == SHAPE and "31 bits" in str(e.value), str(e.value)


def test_softmax():
    refused(B.biv_softmax, f32(BIG, 1), f32(BIG, 1), 1.0)
    refused(B.biv_softmax, f32(1, BIG), f32(1, BIG), 1.0)
    refused(B.biv_softmax, f32(1, BIG), f32(1, BIG), 1.0, V=BIG)


def test_gemm_bias_act():
    refused(B.biv_gemm_bias_act, bf(BIG, 64), bf(64, 64), bf(BIG, 64))
    refused(B.biv_gemm_bias_act, bf(4, 64), bf(BIG, 64), bf(4, BIG))
    refused(B.biv_gemm_bias_act, bf(4, BIG), bf(8, BIG), bf(4, 8))


def test_paged_calls():
    pool, q = bf(9, 2, 16, 64), bf(8, 4, 64)
    write = dict(qkv=bf(8, 8 * 64), q_out=q, k_pages=pool, v_pages=pool, page_table=i32(2, 3), row_slot=i32(8), row_pos=i32(8),
                 theta=1e4, K=8)
    attn = dict(q=q, k_pages=pool, v_pages=pool, page_table=i32(2, 3), row_slot=i32(8), row_pos=i32(8), o=q, rows_per_group=8,
                workspace=torch.empty(64, dtype=torch.uint8, device="meta"))
    large = bf(BIG, 2, 16, 64)
    for fn, args, own in ((B.biv_rope_kv_write_paged, write, dict(K=BIG)), (B.biv_decode_attn_paged, attn, dict(rows_per_group=BIG))):
        refused(fn, **{**args, **own})
        refused(fn, **{**args, "k_pages": large, "v_pages": large})
        refused(fn, **{**args, "page_table": i32(BIG, 3)})
        refused(fn, **{**args, "page_table": i32(2, BIG)})
    refused(B.biv_rope_kv_write_paged, **{**write, "qkv": bf(BIG, 512), "q_out": bf(BIG, 4, 64), "row_slot": i32(BIG), "row_pos": i32(BIG)})
    refused(B.biv_decode_attn_paged, **{**attn, "q": bf(BIG, 4, 64), "o": bf(BIG, 4, 64), "row_slot": i32(BIG), "row_pos": i32(BIG)})
    refused(B.biv_decode_attn_paged_workspace_size, BIG, 4, 64, 3, 16)
    refused(B.biv_decode_attn_paged_workspace_size, 8, 4, 64, BIG, 16)


def test_verify_sample():
    def call(N, K, V):
        B.biv_verify_sample(f32(N * (K + 1), V), None, i32(N, K), f32(N, K), f32(N), i32(N), i32(N, K + 1), i32(N), i32(N))
    refused(call, BIG, 1, 1)
    refused(call, 2, 3, BIG)
    refused(call, 1, BIG, 4)
