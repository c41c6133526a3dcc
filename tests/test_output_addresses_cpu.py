"""Outputs at the address of an input or of another output are refused on the host, each pair of them (error paths only:
no call reaches the HIP runtime)."""
import pytest

import fp8_w8a8_quantized_quantize_amd as fp8
from fp8_w8a8_quantized_quantize_amd import FP8_ERR_INVALID_ARGUMENT, FP8_KV_F32, FP8_OK
from tests.test_expert_rows_abi_cpu import COMBINE, GEMM, GRAD, GROUPED, PERMUTE, QUANT, SORT, call

BASE = {  # every buffer at an address of its own
    "fp8_moe_sort": (SORT, "ids", "offsets row_token row_of"),
    "fp8_moe_permute": (PERMUTE, "x row_of s_tok", "out s_out"),
    "fp8_moe_combine": (COMBINE, "y row_of weights", "out"),
    "fp8_moe_combine_grad": (GRAD, "dout row_of weights", "dy dw"),
    "fp8_gemm_scaled_act": (GEMM, "qa s_tok qw s_ch bias", "y"),
    "fp8_gemm_grouped_scaled_act": (GROUPED, "qa s_tok row_token offsets qw s_ch bias", "y"),
    "fp8_act_quantize": (QUANT, "h live", "q scales"),
}


def own_addresses(name):
    base, ins, outs = BASE[name]
    return {k: 0x100000 * (i + 1) for i, k in enumerate((ins + " " + outs).split())}


PAIRS = [(n, o, x) for n, (_, ins, outs) in BASE.items() for o in outs.split() for x in (ins + " " + outs).split() if x != o]


@pytest.mark.parametrize("name,out,other", PAIRS, ids=str)
def test_refused(name, out, other):
    at = own_addresses(name)
    at[out] = at[other]
    assert call(BASE[name][0], getattr(fp8.lib(), name), **at) == FP8_ERR_INVALID_ARGUMENT


def test_gradient_of_the_weights_at_the_rows():
    at = own_addresses("fp8_moe_combine_grad")
    for kw in (dict(y=at["dw"]), dict(y=at["dw"], dy=0), dict(dw=at["weights"], dy=0)):
        assert call(GRAD, fp8.lib().fp8_moe_combine_grad, **{**at, **kw}) == FP8_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("name,empty", [
    ("fp8_moe_permute", dict(T=0)), ("fp8_moe_combine", dict(T=0)), ("fp8_moe_combine_grad", dict(T=0)),
    ("fp8_gemm_scaled_act", dict(M=0)), ("fp8_gemm_grouped_scaled_act", dict(R=0)), ("fp8_act_quantize", dict(rows=0))], ids=str)
def test_nothing_to_write_is_no_overlap(name, empty):
    same = dict.fromkeys(own_addresses(name), 0x100000)
    if name == "fp8_act_quantize":
        same["live"] = 0
    assert call(BASE[name][0], getattr(fp8.lib(), name), **same, **empty) == FP8_OK


def test_an_fp32_product_may_not_replace_its_bias():
    at = own_addresses("fp8_gemm_scaled_act")
    assert call(GEMM, fp8.lib().fp8_gemm_scaled_act, **{**at, "y": at["bias"]}, residual=0, yt=FP8_KV_F32, M=1) == \
        FP8_ERR_INVALID_ARGUMENT
