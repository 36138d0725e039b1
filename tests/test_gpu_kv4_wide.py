"""Attention over the 4-bit cache with block tables much wider than the sequences, and heads of
256 over lengths that fill the device."""
import pytest

from test_gpu_kv4 import attend, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Tq,HQ,HK,D,page", [(1, 16, 2, 128, 64), (4, 8, 2, 64, 16), (8, 16, 2, 256, 128)])
def test_tables_much_wider_than_the_sequences(Tq, HQ, HK, D, page):
    """Tables for 32768 tokens over sequences of up to 300, with weights: the scores that go
    between the two kernels lie that far apart."""
    check(*attend([300, 1, 0, 129, 17, 64, 255, 2], Tq, HQ, HK, D, page, width=32768 // page, seed=Tq))


@pytest.mark.parametrize("lens,Tq,HQ,HK", [([6600, 3000, 4100, 1, 900, 5000], 1, 16, 2),
                                           ([3000, 2000, 2500], 8, 16, 2), ([4000], 16, 8, 1),
                                           ([700] * 40, 2, 24, 8)])
def test_heads_of_256(lens, Tq, HQ, HK):
    check(*attend(lens, Tq, HQ, HK, 256, 64, seed=HQ))
