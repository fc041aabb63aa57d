"""Loads from tensor memory fill their registers some time after they are issued.  The wait for them has to
name those registers as its operands: arithmetic on them that does not depend on the wait may be scheduled
before it."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_diffusion_speculative_fc_gb300", "csrc")


def test_every_wait_for_tensor_memory_names_its_registers():
    waits = 0
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for m in re.finditer(r'asm volatile\(\s*"tcgen05\.wait::ld', text):
            waits += 1
            # in the statement's own operands, or in those of the statements right behind it
            assert '"+r"' in text[m.start():m.start() + 220], (name, text[:m.start()].count("\n") + 1)
    assert waits > 0
