"""The largest sizes that the operators of sgemm_decode.h take, on a CPU-only machine: what lies past
them is refused on the host.  (Calls that would be taken are made with no rows, which return before
the library touches a device.)
"""
from __future__ import annotations

import pytest

import bf16_skinny_gemm_gb300 as sk
from bf16_skinny_gemm_gb300 import build as skbuild
from bf16_skinny_gemm_gb300 import decode

A = 1 << 40  # pointers that are never dereferenced, far apart


@pytest.fixture(scope="module", autouse=True)
def built():
    skbuild.build()


def norm(D, T, form=0):
    groups = -(-D // 128) if form == 2 else 1
    return decode._fn("sgemm_bf16_add_rmsnorm")(
        decode._NORM.pack(A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A if form else 0, D, D, D, D, groups, T, D, form, 1e-6, 0), None)


@pytest.mark.parametrize("form", [0, 1, 2])
@pytest.mark.parametrize("D", [(1 << 30) + 1, (1 << 31) - 4096, (1 << 31) - 1024, (1 << 31) - 128, (1 << 31) - 1])
def test_norm_refuses_rows_whose_columns_pass_its_counters(D, form):
    """The loop over a long row's columns adds up to 4096 to a 32-bit count below D, and the
    groups' number adds 127 to D."""
    assert norm(D, 1, form) == sk.SGEMM_ERR_UNSUPPORTED_SHAPE
    assert norm(D, 0, form) == sk.SGEMM_ERR_UNSUPPORTED_SHAPE
    assert norm(1 << 30, 0, form) == sk.SGEMM_OK


def test_workspace_of_a_batch_in_which_one_sequence_has_many_tokens():
    """512 sequences of 128 heads, of up to 32768 tokens each: 2^31 rows if all had as many, which is
    more than a call takes, but the call may have far fewer."""
    try:
        assert 0 <= sk.sgemm_latent_attention_workspace(512, 128, 512, 64, 64, 1000, 32768) <= sk.LATENT_WORKSPACE_MAX
    except sk.SgemmError as e:
        assert e.status in (sk.SGEMM_ERR_UNSUPPORTED_DEVICE, sk.SGEMM_ERR_CUDA)
    for batch, max_q in ((-1, 4), (4, 0), (4, -1)):
        with pytest.raises(sk.SgemmError) as e:
            sk.sgemm_latent_attention_workspace(batch, 128, 512, 64, 64, 1000, max_q)
        assert e.value.status == sk.SGEMM_ERR_INVALID_ARG
