"""The block operators' calls refuse bad arguments before anything is launched
(no GPU is needed: the checks come before the device is asked)."""
import pytest

from communication_overlap_gb300 import fo

ARG, UNSUP = fo.FO_ERR_ARG, fo.FO_ERR_UNSUPPORTED


def refused(status, call, *args):
    with pytest.raises(fo.FoError) as e:
        call(*args)
    assert e.value.status == status


ROUTE = dict(desc={}, logits=64, type=1, tokens=4, row_stride=8, bias=64, ids=64, weights=64,
             row_token=64, row_slot=64, token_row=64, expert_first=64, expert_rows=64,
             workspace=64, dev_status=64, stream=0)
DESC = dict(experts=8, top_k=2, renormalize=True, capacity=0, score=1, groups=4, top_groups=2,
            group_top=2, scale=1.0)


def route_args(base, bad):
    args = {**base, **{k: v for k, v in bad.items() if k in base}}
    args["desc"] = fo.make_route_desc(**{**DESC, **{k: v for k, v in bad.items() if k in DESC}})
    return args.values()


BAD_DESC = [
    dict(experts=0), dict(experts=9), dict(top_k=0), dict(top_k=5), dict(score=2), dict(score=-1),
    dict(groups=0), dict(groups=3), dict(groups=8, top_groups=1), dict(top_groups=0),
    dict(top_groups=5), dict(group_top=0), dict(group_top=3), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("inf")), dict(scale=float("nan")), dict(capacity=-1),
    dict(experts=1026, groups=2, row_stride=2000), dict(experts=66, groups=33, row_stride=99),
]


@pytest.mark.parametrize("bad", BAD_DESC + [
    dict(logits=0), dict(ids=0), dict(weights=0), dict(row_token=0), dict(row_slot=0),
    dict(token_row=0), dict(expert_first=0), dict(expert_rows=0), dict(workspace=0),
    dict(dev_status=0), dict(logits=66), dict(bias=66), dict(workspace=72), dict(tokens=-1),
    dict(row_stride=7), dict(type=2),
])
def test_route_refuses(bad):
    refused(ARG, fo.fo_moe_route_scored, *route_args(ROUTE, bad))


BACK = dict(desc={}, logits=64, type=1, tokens=4, row_stride=8, ids=64, weights=64, dweights=64,
            dlogits=64, dlogits_stride=8, stream=0)


@pytest.mark.parametrize("bad", BAD_DESC + [
    dict(logits=0), dict(ids=0), dict(weights=0), dict(dweights=0), dict(dlogits=0),
    dict(dlogits=66), dict(dlogits_stride=7), dict(row_stride=7), dict(tokens=-1), dict(type=2),
])
def test_route_backward_refuses(bad):
    refused(ARG, fo.fo_moe_route_scored_backward, *route_args(BACK, bad))


def test_route_backward_of_nothing_and_of_too_much():
    fo.fo_moe_route_scored_backward(*route_args(BACK, dict(tokens=0)))
    refused(UNSUP, fo.fo_moe_route_scored_backward, *route_args(BACK, dict(tokens=1 << 31)))
    refused(UNSUP, fo.fo_moe_route_scored, *route_args(ROUTE, dict(tokens=1 << 31)))


COMBINE = dict(rows=64, type=0, table_rows=8, hidden=16, row_stride=16, token_row=64, weights=64,
               tokens=4, top_k=2, y=64, y_type=0, y_stride=16, dev_status=64, stream=0)


@pytest.mark.parametrize("bad", [
    dict(rows=0), dict(token_row=0), dict(y=0), dict(dev_status=0), dict(rows=65), dict(y=65),
    dict(y_type=1, y=66), dict(token_row=66), dict(weights=66), dict(dev_status=66), dict(type=2),
    dict(y_type=3), dict(table_rows=-1), dict(hidden=-1), dict(tokens=-1), dict(top_k=0),
    dict(top_k=33), dict(row_stride=15), dict(y_stride=15),
])
def test_combine_refuses(bad):
    refused(ARG, fo.fo_moe_combine, *{**COMBINE, **bad}.values())


def test_combine_of_nothing_and_of_too_much():
    fo.fo_moe_combine(*{**COMBINE, "tokens": 0, "token_row": 0, "y": 0}.values())
    fo.fo_moe_combine(*{**COMBINE, "hidden": 0}.values())
    for big in (dict(tokens=(1 << 31) - (1 << 19)), dict(table_rows=1 << 31),
                dict(hidden=1 << 31, row_stride=1 << 31, y_stride=1 << 31, dy_stride=1 << 31,
                     drows_stride=1 << 31)):
        for call, args in ((fo.fo_moe_combine, COMBINE),
                           (fo.fo_moe_combine_backward, COMBINE_BACK)):
            refused(UNSUP, call, *{**args, **{k: v for k, v in big.items() if k in args}}.values())


COMBINE_BACK = dict(dy=64, dy_type=0, dy_stride=16, rows=64, type=0, table_rows=8, hidden=16,
                    row_stride=16, token_row=64, row_token=64, weights=64, tokens=4, top_k=2,
                    drows=64, drows_stride=16, dweights=64, dev_status=64, stream=0)


@pytest.mark.parametrize("bad", [
    dict(dy=0), dict(rows=0), dict(token_row=0), dict(row_token=0), dict(drows=0),
    dict(dev_status=0), dict(dy=65), dict(drows=65), dict(rows=65), dict(dweights=66),
    dict(row_token=66), dict(token_row=66), dict(type=2), dict(dy_type=2), dict(table_rows=-1),
    dict(hidden=-1), dict(tokens=-1), dict(top_k=0), dict(top_k=33), dict(row_stride=15),
    dict(dy_stride=15), dict(drows_stride=15),
])
def test_combine_backward_refuses(bad):
    refused(ARG, fo.fo_moe_combine_backward, *{**COMBINE_BACK, **bad}.values())


def test_checkpoint_sizes_that_do_not_fit():
    for inter in ((1 << 62) - 31, (1 << 62) - 32, (1 << 61) - 31, 1 << 61):
        for rows in (1, 2, 3):
            refused(ARG, fo.fo_checkpoint_sizes, rows, inter)
    n = (1 << 60) - 32
    assert fo.fo_checkpoint_sizes(1, n) == (2 * n, n // 16)


def test_checkpoint_sizes():
    assert fo.fo_checkpoint_sizes(3, 33) == (3 * 2 * 64, 3 * 2 * 2)
    assert fo.fo_checkpoint_sizes(0, 5) == (0, 0) and fo.fo_checkpoint_sizes(5, 0) == (0, 0)
    for bad in ((-1, 1), (1, -1), (1 << 40, 1 << 40), (1, (1 << 63) - 1)):
        refused(ARG, fo.fo_checkpoint_sizes, *bad)


ACT = dict(u=64, type=0, rows=4, inter=16, u_stride=32, act=2, h=64, h_stride=16, codes=64,
           scales=64, stream=0)


@pytest.mark.parametrize("bad", [
    dict(u=0), dict(h=0), dict(codes=0), dict(scales=0), dict(codes=72), dict(u=65), dict(h=65),
    dict(type=1, h=66), dict(type=2), dict(act=3), dict(act=-1), dict(rows=-1), dict(inter=-1),
    dict(u_stride=31), dict(h_stride=15),
])
def test_act_refuses(bad):
    refused(ARG, fo.fo_gated_act, *{**ACT, **bad}.values())


ACT_BACK = dict(dh=64, type=0, rows=4, inter=16, dh_stride=16, act=2, codes=64, scales=64, du=64,
                du_stride=32, stream=0)


@pytest.mark.parametrize("bad", [
    dict(dh=0), dict(du=0), dict(codes=0), dict(scales=0), dict(codes=72), dict(dh=65),
    dict(du=65), dict(type=2), dict(act=3), dict(rows=-1), dict(inter=-1), dict(du_stride=31),
    dict(dh_stride=15),
])
def test_act_backward_refuses(bad):
    refused(ARG, fo.fo_gated_act_backward, *{**ACT_BACK, **bad}.values())


def test_act_of_nothing_and_of_too_much():
    for empty in (dict(rows=0), dict(inter=0)):
        fo.fo_gated_act(*{**ACT, **empty}.values())
        fo.fo_gated_act_backward(*{**ACT_BACK, **empty}.values())
    refused(UNSUP, fo.fo_gated_act, *{**ACT, "rows": 1 << 31}.values())
    refused(UNSUP, fo.fo_gated_act_backward, *{**ACT_BACK, "rows": 1 << 31}.values())


NORM_DESC = dict(tokens=4, hidden=16, type=0, stream_type=0, param_type=0, gates=2, scale=1.0,
                 eps=1e-6)
NORM = dict(desc={}, x=64, x_stride=16, residual=64, residual_stride=16, post_gain=64, gate=64,
            gate_stride=16, pre_gain=64, sum=64, sum_stride=16, y=64, y_stride=16, post_rstd=64,
            pre_rstd=64, stream=0)
NORM_BACK = dict(desc={}, x=64, x_stride=16, residual=64, residual_stride=16, post_gain=64,
                 gate=64, gate_stride=16, pre_gain=64, post_rstd=64, pre_rstd=64, dsum=64,
                 dsum_stride=16, dy=64, dy_stride=16, dx=64, dx_stride=16, dresidual=64,
                 dresidual_stride=16, dpost=64, dgate=64, dpre=64, workspace=64, stream=0)


def norm_args(base, bad):
    args = {**base, **{k: v for k, v in bad.items() if k in base}}
    args["desc"] = fo.make_norm_desc(**{**NORM_DESC,
                                        **{k: v for k, v in bad.items() if k in NORM_DESC}})
    return args.values()


BAD_NORM = [
    dict(tokens=-1), dict(hidden=-1), dict(type=2), dict(type=1), dict(stream_type=2),
    dict(param_type=2), dict(gates=0), dict(gates=3), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(eps=-1.0), dict(eps=float("nan")), dict(x=0), dict(x=65),
    dict(residual=65), dict(post_gain=65), dict(gate=65), dict(pre_gain=65), dict(x_stride=15),
    dict(residual_stride=15), dict(gate_stride=15), dict(post_rstd=0), dict(pre_rstd=0),
    dict(post_rstd=66), dict(pre_rstd=66),
]


@pytest.mark.parametrize("bad", BAD_NORM + [
    dict(y=0), dict(y=65), dict(sum=65), dict(sum_stride=15), dict(y_stride=15),
])
def test_norm_refuses(bad):
    refused(ARG, fo.fo_block_norm, *norm_args(NORM, bad))


@pytest.mark.parametrize("bad", BAD_NORM + [
    dict(dy=0), dict(dy=65), dict(dsum=65), dict(dsum_stride=15), dict(dy_stride=15), dict(dx=0),
    dict(dx=65), dict(dx_stride=15), dict(dresidual=65), dict(dresidual_stride=15), dict(dpost=0),
    dict(dgate=0), dict(dpre=0), dict(dpost=65), dict(dgate=65), dict(dpre=65), dict(workspace=0),
    dict(workspace=72),
])
def test_norm_backward_refuses(bad):
    refused(ARG, fo.fo_block_norm_backward, *norm_args(NORM_BACK, bad))


def test_norm_of_nothing_and_of_too_much():
    fo.fo_block_norm(*norm_args(NORM, dict(tokens=0)))
    fo.fo_block_norm(*norm_args(NORM, dict(hidden=0)))
    for tokens in (1 << 32, (1 << 31) - (1 << 19)):
        refused(UNSUP, fo.fo_block_norm, *norm_args(NORM, dict(tokens=tokens)))
        refused(UNSUP, fo.fo_block_norm_backward, *norm_args(NORM_BACK, dict(tokens=tokens)))
    desc = fo.make_norm_desc(**NORM_DESC)
    assert fo.fo_block_norm_workspace(desc) > 0
    refused(ARG, fo.fo_block_norm_workspace, fo.make_norm_desc(**{**NORM_DESC, "gates": 3}))
    # any size, none among them: the parts of as many workers as there may be
    for hidden in (0, 1, 255, 256, 257, 2752, 8192, 8193, 100000):
        desc = fo.make_norm_desc(**{**NORM_DESC, "tokens": 1 << 20, "hidden": hidden})
        assert fo.fo_block_norm_workspace(desc) >= (8 << 20 if hidden else 16)
    fo.fo_block_norm_backward(*norm_args(NORM_BACK, dict(hidden=0)))
