"""Numbers given as sampling settings, on the CPU: a temperature that only its rounding to f32
makes 0 is out of range, as it is without the rounding, and not the greedy choice."""
import pytest


@pytest.fixture(scope="module")
def head():
    import q5_lm_head_gb300 as mlh
    h = mlh.LMHead.__new__(mlh.LMHead)
    h.device, h.n_rows, h.k, h.max_batch, h.fmt, h.block_bytes, h.handle = 0, 8, 256, 1, "q5_k", 176, None
    return h


@pytest.mark.parametrize("temperature", [1e-50, -1e-50, 5e-324])
def test_temperature_that_rounds_to_nothing(head, temperature):
    with pytest.raises(ValueError, match="temperature"):
        head._sampling(1, temperature, 0, 1.0, 0.0)


@pytest.mark.parametrize("temperature", [0, 0.0, -0.0, 1, 0.75, 2.0 ** -20, 1e-30])
def test_other_numbers_go_on(head, temperature):
    """In range, or for the call itself to refuse."""
    how = head._sampling(1, temperature, 3, 0.5, 0.25)
    assert how.temperature == pytest.approx(temperature, rel=2.0 ** -24)
    assert (how.top_k, how.top_p, how.min_p) == (3, 0.5, 0.25) and not how.temperatures
