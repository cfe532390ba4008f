"""The example decoder's refusals, on the host."""
import pytest

torch = pytest.importorskip("torch")


def test_generate_refuses_prompts_that_do_not_fit():
    from weight_only_int4_02_gb300 import serve
    prompt = lambda n: torch.zeros(n, dtype=torch.int64)
    for prompts, steps, max_len in (([prompt(60), prompt(3)], 6, 64), ([prompt(65)], 1, 64), ([prompt(4), prompt(0)], 2, 64), ([], 2, 64)):
        with pytest.raises(ValueError):
            serve.generate(None, prompts, steps, max_len=max_len)
