"""Sizes at which the layer operators' launches and addresses end, checked on
the host (fake addresses, never dereferenced)."""
import pytest

from test_layer_abi import OK, TOO_LARGE, at, ssm, ssm_step


def far(*names):
    return {k: at(0) + (i << 45) for i, k in enumerate(names)} | dict(z=0, D=0, bias=0)


@pytest.mark.parametrize("want,H,P,S_", [
    (TOO_LARGE, 65536, 64, 128),  # B and C: rows of 2^23 elements
    (OK, 65535, 64, 128),
    (TOO_LARGE, 65536, 128, 64),  # x and out
    (OK, 65535, 128, 64)])
def test_packed_rows_of_a_prompt_stay_below_their_strides_bound(want, H, P, S_):
    # rows are less than 2^23 elements apart, whether a stride says so or not
    assert ssm(N=1, T=32, H=H, G=H, P=P, S_=S_, s0=0, fin=0, **far("x", "B", "C", "dt", "A", "out", "cu")) == want


def test_single_tokens_take_any_number_of_groups():
    assert ssm_step(n=1, T=1, H=65536, G=65536, P=64, S_=128, size=1,
                    **far("x", "B", "C", "dt", "A", "out", "pool", "idx")) == OK
