"""Refusals of the expert and adapter entry points: every invalid argument is answered with its
documented status before anything reaches the device (no GPU needed, no kernel is launched)."""
import os

import pytest

import bit_weight_quantization_amd as hq
import bit_weight_quantization_amd.build  # noqa: F401  (hq.build)

FAKE = 1 << 20  # a 1 MiB-aligned fake device address: never dereferenced, validation fails first
INV, UNS, ALN = hq.HQQ_ERR_INVALID_ARG, hq.HQQ_ERR_UNSUPPORTED, hq.HQQ_ERR_ALIGNMENT


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(hq.LIB_PATH):  # build only when nothing is built
        hq.build.build()
    return hq.load_library()


CALLS = {
    "hqq_expert_sort": dict(ids_i32=FAKE, tokens=4, topk=2, experts=8, order_i32=FAKE,
                            position_i32=FAKE, offsets_i32=FAKE, workspace=0),
    "hqq_expert_gather": dict(X=FAKE, dtype=0, tokens=4, topk=2, width=64, position_i32=FAKE, Xs=FAKE),
    "hqq_expert_combine": dict(Ys=FAKE, dtype=0, tokens=4, topk=2, width=64, position_i32=FAKE,
                               weights_f32=FAKE, out=FAKE),
    "hqq_expert_combine_backward": dict(dOut=FAKE, Ys=FAKE, dtype=0, tokens=4, topk=2, width=64,
                                        position_i32=FAKE, weights_f32=FAKE, dYs=FAKE,
                                        dweights_f32=FAKE),
    "hqq_matmul_experts": dict(X_f16=FAKE, rows=8, K=128, order_i32=FAKE, topk=2, offsets_i32=FAKE,
                               experts=4, packed_codes=FAKE, scale_f16=FAKE, zero_f16=FAKE, N=16,
                               nbits=4, group_size=64, Y=FAKE, out_f32=0, workspace=0),
    "hqq_matmul_experts_backward": dict(dY_f16=FAKE, rows=8, N=16, offsets_i32=FAKE, experts=4,
                                        packed_codes=FAKE, scale_f16=FAKE, zero_f16=FAKE, K=128,
                                        nbits=4, group_size=64, dX=FAKE, out_f32=0, workspace=FAKE),
    "hqq_matmul_backward": dict(dY_f16=FAKE, M=8, N=4096, packed_codes=FAKE, scale_f16=FAKE,
                                zero_f16=FAKE, K=128, nbits=4, group_size=64, dX=FAKE, out_f32=0,
                                workspace=FAKE),
    "hqq_adapters": dict(X=FAKE, dtype=0, M=4, K=128, A=FAKE, B=FAKE, N=16, rank=8, adapters=2,
                         ids_i32=FAKE, scales_f32=FAKE, base=0, base_f32=0, Y=FAKE, out_f32=0,
                         workspace=FAKE),
    "hqq_adapters_backward": dict(dY=FAKE, X=FAKE, dtype=0, M=4, K=128, A=FAKE, B=FAKE, N=16, rank=8,
                                  adapters=2, ids_i32=FAKE, scales_f32=FAKE, base=0, base_f32=0,
                                  dX=FAKE, out_f32=0, dA_f32=FAKE, dB_f32=FAKE, workspace=FAKE),
    "hqq_matmul_adapters": dict(X_f16=FAKE, M=4, K=128, packed_codes=FAKE, scale_f16=FAKE,
                                zero_f16=FAKE, N=16, nbits=4, group_size=64, A_f16=FAKE, B_f16=FAKE,
                                rank=8, adapters=2, ids_i32=FAKE, scales_f32=FAKE, Y=FAKE, out_f32=0,
                                workspace=FAKE),
    "hqq_matmul_adapters_backward": dict(dY_f16=FAKE, X_f16=FAKE, M=4, K=128, packed_codes=FAKE,
                                         scale_f16=FAKE, zero_f16=FAKE, N=16, nbits=4, group_size=64,
                                         A_f16=FAKE, B_f16=FAKE, rank=8, adapters=2, ids_i32=FAKE,
                                         scales_f32=FAKE, dX=FAKE, out_f32=0, dA_f32=FAKE,
                                         dB_f32=FAKE, workspace=FAKE),
}

BAD = {
    "hqq_matmul_adapters": [
        (dict(nbits=5), UNS), (dict(group_size=48), UNS), (dict(K=96), INV),
        (dict(K=48, group_size=16), UNS), (dict(K=1 << 25), INV), (dict(M=-1), INV),
        (dict(M=2000001), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(rank=12), UNS),
        (dict(rank=512), UNS), (dict(adapters=0), INV), (dict(adapters=1025), UNS),
        (dict(X_f16=0), INV), (dict(packed_codes=0), INV), (dict(A_f16=0), INV), (dict(B_f16=0), INV),
        (dict(ids_i32=0), INV), (dict(scales_f32=0), INV), (dict(Y=0), INV), (dict(workspace=0), INV),
        (dict(out_f32=2), INV), (dict(X_f16=FAKE + 8), ALN), (dict(packed_codes=FAKE + 8), ALN),
        (dict(zero_f16=FAKE + 1), ALN), (dict(A_f16=FAKE + 4), ALN), (dict(ids_i32=FAKE + 2), ALN),
        (dict(Y=FAKE + 2, out_f32=1), ALN), (dict(workspace=FAKE + 64), ALN)],
    "hqq_matmul_adapters_backward": [
        (dict(nbits=7), UNS), (dict(K=100), INV), (dict(M=2000001), INV), (dict(rank=4), UNS),
        (dict(dY_f16=0), INV), (dict(X_f16=0), INV), (dict(scale_f16=0), INV), (dict(dX=0), INV),
        (dict(dA_f32=0), INV), (dict(dB_f32=0), INV), (dict(workspace=0), INV),
        (dict(M=0, dA_f32=0), INV), (dict(dY_f16=FAKE + 1), ALN), (dict(dB_f32=FAKE + 8), ALN),
        (dict(packed_codes=FAKE + 2), ALN), (dict(workspace=FAKE + 4), ALN)],
    "hqq_expert_sort": [
        (dict(tokens=-1), INV), (dict(topk=0), INV), (dict(topk=-3), INV), (dict(experts=0), INV),
        (dict(experts=1025), UNS), (dict(tokens=1 << 31, topk=1), INV),
        (dict(tokens=1 << 30, topk=4), INV), (dict(ids_i32=0), INV), (dict(order_i32=0), INV),
        (dict(position_i32=0), INV), (dict(offsets_i32=0), INV), (dict(ids_i32=FAKE + 2), ALN),
        (dict(offsets_i32=FAKE + 1), ALN), (dict(tokens=5000), INV),  # needs a workspace
        (dict(tokens=5000, workspace=FAKE + 2), ALN)],
    "hqq_expert_gather": [
        (dict(dtype=3), UNS), (dict(dtype=-1), UNS), (dict(tokens=-1), INV), (dict(topk=0), INV),
        (dict(width=-1), INV), (dict(width=1 << 61), INV), (dict(X=0), INV), (dict(Xs=0), INV),
        (dict(position_i32=0), INV), (dict(X=FAKE + 1), ALN), (dict(Xs=FAKE + 2, dtype=2), ALN),
        (dict(position_i32=FAKE + 2), ALN)],
    "hqq_expert_combine": [
        (dict(dtype=7), UNS), (dict(tokens=-1), INV), (dict(topk=0), INV), (dict(Ys=0), INV),
        (dict(out=0), INV), (dict(position_i32=0), INV), (dict(weights_f32=FAKE + 2), ALN),
        (dict(Ys=FAKE + 1), ALN), (dict(out=FAKE + 2, dtype=2), ALN)],
    "hqq_expert_combine_backward": [
        (dict(dtype=5), UNS), (dict(topk=-1), INV), (dict(dOut=0), INV), (dict(Ys=0), INV),
        (dict(dYs=0), INV), (dict(position_i32=0), INV), (dict(dweights_f32=FAKE + 2), ALN),
        (dict(weights_f32=FAKE + 1), ALN), (dict(dYs=FAKE + 1), ALN)],
    "hqq_matmul_experts": [
        (dict(nbits=5), UNS), (dict(group_size=48), UNS), (dict(K=120), INV),
        (dict(K=48, group_size=16), UNS), (dict(experts=0), INV), (dict(experts=2000), UNS),
        (dict(rows=-1), INV), (dict(rows=8000001), INV), (dict(out_f32=2), INV), (dict(topk=0), INV),
        (dict(N=1 << 60), INV), (dict(X_f16=0), INV), (dict(packed_codes=0), INV),
        (dict(scale_f16=0), INV), (dict(zero_f16=0), INV), (dict(Y=0), INV),
        (dict(offsets_i32=0), INV), (dict(X_f16=FAKE + 8), ALN), (dict(packed_codes=FAKE + 4), ALN),
        (dict(scale_f16=FAKE + 1), ALN), (dict(offsets_i32=FAKE + 2), ALN),
        (dict(order_i32=FAKE + 2), ALN), (dict(Y=FAKE + 2, out_f32=1), ALN),
        (dict(rows=400, K=1024), INV), (dict(rows=400, K=1024, workspace=FAKE + 8), ALN)],
    "hqq_matmul_experts_backward": [
        (dict(nbits=1), UNS), (dict(group_size=256), UNS), (dict(K=96), INV), (dict(experts=-1), INV),
        (dict(experts=1025), UNS), (dict(rows=8000001), INV), (dict(out_f32=-1), INV),
        (dict(dY_f16=0), INV), (dict(dX=0), INV), (dict(offsets_i32=0), INV),
        (dict(packed_codes=0), INV), (dict(dY_f16=FAKE + 1), ALN), (dict(packed_codes=FAKE + 8), ALN),
        (dict(dX=FAKE + 1), ALN), (dict(N=8192, workspace=0), INV),
        (dict(N=8192, workspace=FAKE + 8), ALN)],
    "hqq_matmul_backward": [
        (dict(nbits=6), UNS), (dict(group_size=8), UNS), (dict(K=100), INV),
        (dict(K=48, group_size=16), UNS), (dict(M=-1), INV), (dict(M=8000001), INV),
        (dict(N=-1), INV), (dict(out_f32=3), INV), (dict(dY_f16=0), INV), (dict(dX=0), INV),
        (dict(scale_f16=0), INV), (dict(dY_f16=FAKE + 1), ALN), (dict(zero_f16=FAKE + 1), ALN),
        (dict(workspace=0), INV), (dict(workspace=FAKE + 4), ALN)],
    "hqq_adapters": [
        (dict(dtype=2), UNS), (dict(dtype=-1), UNS), (dict(M=-1), INV), (dict(M=2000001), INV),
        (dict(N=0), INV), (dict(K=0), INV), (dict(K=100), UNS), (dict(rank=0), INV),
        (dict(rank=12), UNS), (dict(rank=264), UNS), (dict(adapters=0), INV),
        (dict(adapters=1025), UNS), (dict(N=1 << 58), INV), (dict(X=0), INV), (dict(A=0), INV),
        (dict(B=0), INV), (dict(ids_i32=0), INV), (dict(scales_f32=0), INV), (dict(Y=0), INV),
        (dict(workspace=0), INV), (dict(base_f32=2), INV), (dict(out_f32=2), INV),
        (dict(base=FAKE, base_f32=1), INV),  # in place over another type
        (dict(X=FAKE + 8), ALN), (dict(A=FAKE + 8), ALN), (dict(B=FAKE + 2), ALN),
        (dict(ids_i32=FAKE + 1), ALN), (dict(scales_f32=FAKE + 2), ALN), (dict(base=FAKE + 1), ALN),
        (dict(Y=FAKE + 2, out_f32=1), ALN), (dict(workspace=FAKE + 128), ALN)],
    "hqq_adapters_backward": [
        (dict(dtype=2), UNS), (dict(M=2000001), INV), (dict(K=4), UNS), (dict(rank=7), UNS),
        (dict(adapters=1025), UNS), (dict(dY=0), INV), (dict(X=0), INV), (dict(dX=0), INV),
        (dict(dA_f32=0), INV), (dict(dB_f32=0), INV), (dict(workspace=0), INV),
        (dict(M=0, dB_f32=0), INV), (dict(base=FAKE, out_f32=1), INV), (dict(dY=FAKE + 1), ALN),
        (dict(dA_f32=FAKE + 8), ALN), (dict(dB_f32=FAKE + 4), ALN), (dict(workspace=FAKE + 16), ALN)],
}


@pytest.mark.parametrize("name,kw,status",
                         [(n, kw, st) for n, cases in BAD.items() for kw, st in cases])
def test_invalid_arguments_are_refused(name, kw, status):
    assert getattr(hq, name)(**{**CALLS[name], **kw}) == status


def test_calls_without_work_are_no_ops():
    none = dict(X_f16=0, packed_codes=0, scale_f16=0, zero_f16=0, Y=0, offsets_i32=0, order_i32=0)
    assert hq.hqq_matmul_experts(**{**CALLS["hqq_matmul_experts"], **none, "rows": 0}) == hq.HQQ_OK
    assert hq.hqq_matmul_backward(**{**CALLS["hqq_matmul_backward"], "M": 0, "dX": 0}) == hq.HQQ_OK
    assert hq.hqq_expert_gather(**{**CALLS["hqq_expert_gather"], "tokens": 0, "X": 0}) == hq.HQQ_OK
    assert hq.hqq_expert_combine(**{**CALLS["hqq_expert_combine"], "width": 0, "Ys": 0}) == hq.HQQ_OK
    assert hq.hqq_adapters(**{**CALLS["hqq_adapters"], "M": 0, "X": 0}) == hq.HQQ_OK


def test_workspace_sizes():
    assert hq.hqq_expert_sort_workspace_bytes(4096, 1, 8) == 0
    assert hq.hqq_expert_sort_workspace_bytes(4097, 1, 8) > 0
    assert hq.hqq_expert_sort_workspace_bytes(0, 1, 8) == 0
    for bad in ((-1, 1, 8), (1, 0, 8), (1, 1, 0), (1, 1, 1025), (1 << 31, 1, 8)):
        assert hq.hqq_expert_sort_workspace_bytes(*bad) == -1
    assert hq.hqq_matmul_backward_workspace_bytes(8192, 4096, 4096) == 0   # tiles enough
    assert hq.hqq_matmul_backward_workspace_bytes(8, 4096, 1024) > 0       # few rows: N is split
    assert hq.hqq_matmul_backward_workspace_bytes(8, 512, 1024) == 0       # too short to split
    assert hq.hqq_matmul_backward_workspace_bytes(-1, 4, 32) == -1
    assert hq.hqq_matmul_experts_backward_workspace_bytes(16, 4096, 1024, 0) == -1
    assert hq.hqq_matmul_experts_backward_workspace_bytes(16, 1 << 60, 1024, 8) == -1
    assert hq.hqq_adapters_workspace_bytes(1, 4096, 4096, 16, 8) >= 16 * 4
    assert hq.hqq_adapters_workspace_bytes(1, 4096, 4096, 12, 8) == -1
    small = hq.hqq_adapters_backward_workspace_bytes(64, 4096, 4096, 16, 1)
    assert hq.hqq_adapters_backward_workspace_bytes(64, 4096, 4096, 16, 8) > small > 0


def test_tensor_arguments_are_checked_without_a_device():
    torch = pytest.importorskip("torch")
    ids = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        hq.expert_sort(ids, 4)
    with pytest.raises(ValueError, match="int32"):
        hq.expert_sort(ids.long(), 4)
    with pytest.raises(ValueError, match="topk"):
        hq.expert_sort(ids.view(1, 2, 2), 4)
    route = hq.ExpertOrder(ids.view(-1), ids.view(-1), torch.zeros(5, dtype=torch.int32), 2, 2, 4)
    with pytest.raises(ValueError, match="float16, bfloat16 or float32"):
        hq.expert_gather(torch.zeros((2, 8), dtype=torch.float64), route)
    q = hq.QuantizedWeight(packed=ids, scale=ids, zero=ids, rows=10, cols=64, nbits=4, group_size=64)
    with pytest.raises(ValueError, match="experts of equal size"):
        hq.matmul_experts(torch.zeros((2, 64), dtype=torch.float16), q, route)
    with pytest.raises(ValueError, match="adapters x rank x K"):
        hq.adapters(torch.zeros(2, 64).half(), torch.zeros(8, 64).half(), torch.zeros(1, 4, 8).half(),
                    ids.view(-1), torch.zeros(1))
