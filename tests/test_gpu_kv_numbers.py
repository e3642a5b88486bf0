"""Reads of one head on both sides of where a job takes four tokens."""

import pytest

from test_gpu_kv import test_reads_of_few_heads as reads_of_few_heads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("hd,T", [(64, 4799), (64, 4802), (128, 4800), (128, 4807), (256, 4801), (256, 6003)])
def test_reads_of_one_head_around_four_tokens_a_job(kind, hd, T):
    reads_of_few_heads(kind, 1, hd, T)
