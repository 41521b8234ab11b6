"""The expert layer's calls refuse bad arguments before anything is launched
(no GPU is needed: the checks come before the device is asked)."""
import ctypes

import pytest

from communication_overlap_gb300 import fo

ARG, UNSUP = fo.FO_ERR_ARG, fo.FO_ERR_UNSUPPORTED


def refused(status, call, *args):
    with pytest.raises(fo.FoError) as e:
        call(*args)
    assert e.value.status == status


def test_mx_sizes():
    assert fo.fo_mx_sizes(1, 1, 1) == (128 * 64, 512)
    assert fo.fo_mx_sizes(3, 129, 128) == (3 * 256 * 64, 3 * 1024)
    assert fo.fo_mx_sizes(0, 5, 5) == (0, 0)
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, -1), (1, 1 << 40, 1 << 40), (1, (1 << 63) - 1, 1)):
        refused(ARG, fo.fo_mx_sizes, *bad)


QUANT = dict(src=64, type=0, batch=1, batch_stride=0, rows=8, cols=64, row_stride=64, transpose=0,
             row_index=0, src_rows=8, codes=64, scales=64, stream=0)


@pytest.mark.parametrize("bad", [
    dict(src=0), dict(codes=0), dict(scales=0), dict(codes=72), dict(scales=68), dict(src=65),
    dict(type=1, src=66), dict(type=2), dict(type=7), dict(rows=-1), dict(cols=-1), dict(batch=-1),
    dict(row_stride=63), dict(transpose=1, row_stride=7), dict(batch_stride=-1),
    dict(row_index=66), dict(row_index=64, transpose=1), dict(row_index=64, batch=2),
    dict(row_index=64, src_rows=-1),
])
def test_quantize_refuses(bad):
    refused(ARG, fo.fo_mx_quantize, *{**QUANT, **bad}.values())


def test_quantize_of_nothing_and_of_too_much():
    for empty in (dict(rows=0), dict(cols=0), dict(batch=0)):
        fo.fo_mx_quantize(*{**QUANT, "row_stride": 64, **empty}.values())
    refused(UNSUP, fo.fo_mx_quantize, *{**QUANT, "rows": 1 << 31}.values())


DEQ = dict(codes=64, scales=64, batch=1, rows=8, cols=64, dst=64, type=0, batch_stride=0,
           row_stride=64, stream=0)


@pytest.mark.parametrize("bad", [
    dict(codes=0), dict(scales=0), dict(dst=0), dict(codes=8), dict(scales=8), dict(dst=65),
    dict(type=1, dst=66), dict(type=2), dict(rows=-1), dict(row_stride=63), dict(batch_stride=-1),
])
def test_dequantize_refuses(bad):
    refused(ARG, fo.fo_mx_dequantize, *{**DEQ, **bad}.values())


GEMM = dict(M=8, N=8, K=64, A_codes=64, A_scales=64, B_codes=64, B_scales=64, n_groups=0,
            group_first=0, group_rows=0, D=64, type=0, row_stride=8, dev_status=64, stream=0)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(A_codes=0), dict(A_scales=0), dict(B_codes=0),
    dict(B_scales=0), dict(A_codes=8), dict(A_scales=8), dict(B_codes=8), dict(B_scales=8),
    dict(D=0), dict(D=65), dict(type=1, D=66), dict(type=2), dict(row_stride=7),
    dict(dev_status=0), dict(dev_status=66), dict(n_groups=-1), dict(n_groups=1025),
    dict(n_groups=1), dict(n_groups=1, group_first=64), dict(group_first=64, group_rows=64),
    dict(n_groups=1, group_first=66, group_rows=64),
])
def test_gemm_refuses(bad):
    refused(ARG, fo.fo_mx_gemm, *{**GEMM, **bad}.values())


def test_gemm_of_nothing_and_of_too_much():
    for empty in (dict(M=0), dict(N=0, row_stride=0)):
        fo.fo_mx_gemm(*{**GEMM, **empty}.values())
    refused(UNSUP, fo.fo_mx_gemm, *{**GEMM, "M": 1 << 31}.values())
    refused(UNSUP, fo.fo_mx_gemm, *{**GEMM, "N": 1 << 24, "row_stride": 1 << 24, "n_groups": 256,
                                    "group_first": 64, "group_rows": 64}.values())


def test_route_sizes():
    rows, ws = fo.fo_moe_route_sizes(100, 8, 2)
    assert rows == (200 + 8 * 127) // 128 * 128 and ws > 0
    assert fo.fo_moe_route_sizes(100, 8, 2, 128)[0] == 1024
    for bad in ((-1, 8, 2), (1, 0, 1), (1, 8, 0), (1, 8, 9), (1, 1025, 2), (1, 64, 33),
                (1, 8, 2, -1)):
        refused(ARG, fo.fo_moe_route_sizes, *bad)
    refused(UNSUP, fo.fo_moe_route_sizes, 1 << 31, 8, 2)
    refused(UNSUP, fo.fo_moe_route_sizes, 1, 8, 2, 1 << 29)


ROUTE = dict(logits=64, type=1, tokens=4, experts=8, row_stride=8, top_k=2, renormalize=1,
             capacity=0, ids=64, weights=64, row_token=64, row_slot=64, token_row=64,
             expert_first=64, expert_rows=64, workspace=64, dev_status=64, stream=0)


@pytest.mark.parametrize("bad", [
    *[{n: 0} for n in ("logits", "ids", "weights", "row_token", "row_slot", "token_row",
                       "expert_first", "expert_rows", "workspace", "dev_status")],
    *[{n: 66} for n in ("logits", "ids", "weights", "row_token", "row_slot", "token_row",
                        "expert_first", "expert_rows", "dev_status")],
    dict(workspace=72), dict(type=2), dict(type=0, logits=65), dict(row_stride=7),
    dict(tokens=-1), dict(top_k=9), dict(capacity=-1),
])
def test_route_refuses(bad):
    refused(ARG, fo.fo_moe_route, *{**ROUTE, **bad}.values())


BACK = dict(logits=64, type=1, tokens=4, experts=8, row_stride=8, top_k=2, renormalize=1, ids=64,
            weights=64, dweights=64, dlogits=64, dlogits_stride=8, stream=0)


@pytest.mark.parametrize("bad", [
    *[{n: 0} for n in ("logits", "ids", "weights", "dweights", "dlogits")],
    *[{n: 66} for n in ("logits", "ids", "weights", "dweights", "dlogits")],
    dict(type=2), dict(row_stride=7), dict(dlogits_stride=7), dict(tokens=-1), dict(top_k=0),
])
def test_route_backward_refuses(bad):
    refused(ARG, fo.fo_moe_route_backward, *{**BACK, **bad}.values())


FEW = dict(tokens=4, hidden=64, inter=64, experts=8, top_k=2)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(tokens=65), dict(hidden=0), dict(hidden=60), dict(inter=0),
    dict(inter=12), dict(experts=0), dict(experts=1025), dict(top_k=0), dict(top_k=9),
    dict(act=3), dict(act=-1), dict(weights=fo.FO_TYPE_F32),
])
def test_few_refuses_descriptions(bad):
    refused(ARG, fo.fo_moe_few_workspace, fo.make_few_desc(**{**FEW, **bad}))


FEW_ARGS = dict(x=64, x_stride=64, router=64, W1=64, W1_scales=0, W2=64, W2_scales=0, y=64,
                y_stride=64, workspace=64, dev_status=64, stream=0)


@pytest.mark.parametrize("bad", [
    *[{n: 0} for n in ("x", "router", "W1", "W2", "y", "workspace", "dev_status")],
    *[{n: 72} for n in ("x", "router", "W1", "W2", "workspace")],
    dict(y=65), dict(dev_status=66), dict(W1_scales=64), dict(W2_scales=64), dict(x_stride=63),
    dict(x_stride=68), dict(y_stride=63),
])
def test_few_refuses(bad):
    d = fo.make_few_desc(**FEW)
    refused(ARG, fo.fo_moe_few, d, *{**FEW_ARGS, **bad}.values())


def test_few_needs_the_scales_of_4_bit_weights():
    d = fo.make_few_desc(**FEW, weights=fo.FO_TYPE_MX4)
    refused(ARG, fo.fo_moe_few, d, *FEW_ARGS.values())
    refused(ARG, fo.fo_moe_few, d, *{**FEW_ARGS, "W1_scales": 64, "W2_scales": 72}.values())
    too_many = fo.make_few_desc(**{**FEW, "inter": 1 << 21, "experts": 1024},
                                weights=fo.FO_TYPE_BF16)
    refused(UNSUP, fo.fo_moe_few, too_many, *FEW_ARGS.values())


def test_null_outputs_of_the_size_queries():
    L = fo.lib()
    assert L.fo_mx_sizes(1, 1, 1, None, None) == fo.FO_OK
    assert L.fo_moe_route_sizes(1, 8, 2, 0, None, None) == fo.FO_OK
    assert L.fo_moe_few_workspace(None, None) == ARG
    d = fo.make_few_desc(**FEW)
    assert L.fo_moe_few_workspace(ctypes.byref(d), None) == ARG
