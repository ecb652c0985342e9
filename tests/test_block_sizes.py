"""Sizes that the C ABI's int does not hold are refused by the binding of
libmoe_block.so: cut to 32 bits they would be small, valid ones.  Views that
repeat one element stand for the tensors, so no memory is needed."""
import pytest
import torch

BF, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
BIG = 1 << 32


@pytest.fixture(scope="module")
def ep():
    import combine_top_expert_amd as ep
    return ep


def v(*shape, dtype=F32):
    return torch.zeros(1, dtype=dtype).expand(*shape)


def calls(ep):
    for T, H in ((BIG + 4, 256), (4, BIG + 256), (BIG, 256), ((1 << 31), 256)):
        x = v(T, H, dtype=BF)
        yield f"norm {T} {H}", lambda x=x, H=H: ep.moe_add_rms_norm(x, None, v(H, dtype=BF), 1e-6, None, x)
        yield f"norm backward {T} {H}", lambda x=x, H=H: ep.moe_add_rms_norm_backward(x, x, v(H, dtype=BF), 1e-6, x, v(H),
                                                                                    v(1 << 20, dtype=U8))
        x8 = v(T, H, dtype=U8)
        yield f"permute {T} {H}", lambda x8=x8, T=T, H=H: ep.moe_permute_fp8(x8, v(T, H // 128), v(T, 2, dtype=I32),
                                                                           v(9, H, dtype=U8), v(9, H // 128))
    yield "permute K", lambda: ep.moe_permute_fp8(v(4, 256, dtype=U8), v(4, 2), v(4, BIG + 2, dtype=I32), v(9, 256, dtype=U8), v(9, 2))
    for T, E, K in ((BIG + 4, 16, 2), (4, BIG + 16, 2), (4, 16, BIG + 2)):
        yield f"route {T} {E} {K}", lambda T=T, E=E, K=K: ep.moe_router_group_topk(v(T, E), K, v(T, K, dtype=I32), v(T, K))
        yield f"route backward {T} {E} {K}", lambda T=T, E=E, K=K: ep.moe_router_group_topk_backward(
            v(T, E), v(T, K, dtype=I32), v(T, K), v(T, E))
    yield "route groups", lambda: ep.moe_router_group_topk(v(4, 16), 2, v(4, 2, dtype=I32), v(4, 2), n_group=BIG + 1)
    yield "route kept groups", lambda: ep.moe_router_group_topk(v(4, 16), 2, v(4, 2, dtype=I32), v(4, 2), n_group=4,
                                                                topk_group=BIG + 2)
    for L, N, K in ((BIG + 2, 128, 256), (2, BIG + 128, 256), (2, 128, BIG + 256)):
        c, s = v(L, N, K // 2, dtype=U8), v(L, N, K // 128)
        yield f"pack {L} {N} {K}", lambda c=c, s=s: ep.moe_pack_w4(c, s, ep.MOE_W4_INT4, c, s)
        yield f"gemv {L} {N} {K}", lambda c=c, s=s, L=L, N=N, K=K: ep.moe_grouped_gemv_w4(
            v(9, K, dtype=BF), None, c, s, ep.MOE_W4_INT4, v(L, dtype=I32), v(L + 1, dtype=I32), ep.MOE_EPI_STORE_G, v(9, N))


def test_sizes_past_32_bits(ep):
    for what, call in calls(ep):
        with pytest.raises(ep.MoEError) as e:
            call()
        assert e.value.status == -2, what


def test_workspace_of_sizes_past_32_bits(ep):
    need = ep.moe_add_rms_norm_backward_workspace_bytes
    assert need(4, 256) > 0
    assert need(BIG + 4, 256) == 0 and need(4, BIG + 256) == 0 and need(-BIG + 4, 256) == 0 and need(4, 256 - BIG) == 0
