"""qkv_rope and kv_append refuse results that overlap the form's arrays, the status or the slots, on the host."""
import ctypes

import pytest

from tests.test_sampled_abi import K, POS, Q, SLOT, ST, U, V, X, append, cache, form, rope, w12  # noqa: F401 (the fixture)


@pytest.mark.parametrize("name", ["q_norm", "k_norm", "inv_freq"])
@pytest.mark.parametrize("out,bytes_", [(Q, 4 * 512 * 2), (K, 4 * 256 * 2), (U, 4 * 256 * 2)])
def test_results_over_the_form(w12, name, out, bytes_):
    size = 4 * (64 if name == "inv_freq" else 128)
    for at in (out.value, out.value + bytes_ - 4, out.value - size + 4):
        assert rope(w12, form(w12, **{name: at})) == 1
        assert w12.lib().w12_last_error().startswith(b"qkv_rope")
        assert append(w12, form(w12, **{name: at})) == 1


@pytest.mark.parametrize("name", ["q_norm", "k_norm", "inv_freq"])
def test_the_cache_over_the_form(w12, name):
    for at in (1 << 30, (1 << 31) + 64):
        assert append(w12, form(w12, **{name: at})) == 1
        assert w12.lib().w12_last_error().startswith(b"kv_append")


@pytest.mark.parametrize("status", [X, POS, SLOT, Q, K, U, V(256), V((3 << 20) + 4 * 512 * 2 - 4)])
def test_the_status_over_another_array(w12, status):
    assert append(w12, status=status) == 1
    assert w12.lib().w12_last_error().startswith(b"kv_append")
