"""The most tokens of one append to the 8-bit cache: a sequence's last block is found from its
tokens, its first place and a block's length in 32 bits.  Refused before any CUDA call."""
from test_fp8_abi_cpu import append, lib  # noqa: F401  (lib: a fixture)


def test_append_refuses_more_tokens_than_its_numbers_hold(lib):
    for T in (2 ** 31 - 31, 2 ** 31 - 1):
        assert append(lib, T=T, Hq=0, q=None, qo=None, s2=0, s4=0) == 2
        assert append(lib, T=T) == 2
