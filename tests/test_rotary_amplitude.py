"""A rotary amplitude is held in float32: one that is zero or infinite there is refused."""
import pytest


@pytest.fixture
def bind(host_lib):
    from paged_kv_decode_10_gb300 import binding
    return binding


@pytest.mark.parametrize("amplitude", [1e39, 3.5e38, 1e-46, 1e-300, float("inf"), -1.0])
def test_amplitudes_outside_float32_are_refused(bind, amplitude):
    with pytest.raises(bind.PkvError):
        bind.Rotary(64, amplitude=amplitude)


@pytest.mark.parametrize("amplitude", [1e-45, 1.2772588722239782, 3.4e38])
def test_amplitudes_inside_it_are_kept(bind, amplitude):
    held = bind.Rotary(64, amplitude=amplitude).table.amplitude
    # one rounding to float32: relative 2^-24, or half its least step, 2^-150
    assert 0 < held < float("inf") and abs(held - amplitude) <= max(2.0**-24 * amplitude, 2.0**-150)
