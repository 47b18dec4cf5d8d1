"""The smallest eps of lora_adamw_step, refused on the host (no GPU, fake pointers)."""
import pytest

from test_abi_training_cpu import ESHAPE, L, P, opt  # noqa: F401 (L is a fixture)


@pytest.mark.parametrize("bits,eps", [(8, 1e-13), (8, 1e-15), (8, 2.0 ** -41), (8, 2.0 ** -126),
                                      (32, 2.0 ** -127), (32, 1e-39)])
def test_eps_out_of_range(L, bits, eps):  # noqa: F811
    scales = {} if bits == 8 else dict(m_scale=None, v_scale=None)
    assert L.lora_adamw_step(opt(L, state_bits=bits, **scales), 1e-3, None, 0.9, 0.999, eps, 0.01,
                             None, None, 0, None) == ESHAPE
