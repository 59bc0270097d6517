"""The order of the loads in the kernels whose waits count them (no GPU: the
sources are compiled to assembly).

A wave waits before a barrier until at most N of its loads are still on their
way, N being the loads to registers that it started after its last load to
LDS.  The other waves read that LDS after the barrier, so between two barriers
no load to registers may be issued before a load to LDS: the wait would let one
to LDS go on."""
import re
import subprocess

import pytest

from param_collectives_amd import build


@pytest.fixture(scope="module")
def segments(tmp_path_factory):
    """{kernel: its instructions between barriers, "L" for a load to LDS and "r"
    for one to registers}, of one source file."""

    def of(source):
        path = tmp_path_factory.mktemp("asm") / "out.s"
        subprocess.run([build.hipcc(), *build.FLAGS, "--offload-device-only", "-S", f"{build.CSRC}/{source}", "-o",
                        str(path)], check=True)
        found, name = {}, None
        for line in path.read_text().splitlines():
            label = re.match(r"(_Z\w+):", line)
            if label:
                name = label.group(1)
                found[name] = [""]
            elif line.startswith(".Lfunc_end"):
                name = None
            elif name:
                op = line.split()[0] if line.split() else ""
                if op == "s_barrier":
                    found[name].append("")
                elif re.match(r"(global|buffer|flat|scratch)_load", op):
                    found[name][-1] += "L" if re.search(r"\blds\b|_lds_", line) else "r"
        return found

    return of


def test_few_tokens_states_before_weights(segments):
    kernels = {n: s for n, s in segments("vocab_loss.hip").items() if "few_logits_kernel" in n}
    assert len(kernels) == 4
    for name, parts in kernels.items():
        fragments = int(re.search(r"few_logits_kernelILi(\d)E", name).group(1))
        # the first block's, two in the loop and one before the last block
        assert [p for p in parts if p.endswith("L" * 2 * fragments + "r" * 8)], name
        assert sum("L" in p for p in parts) >= 4, (name, parts)
        for p in parts:
            assert "rL" not in p, (name, parts)


def test_weight_gradient_rows_before_codes(segments):
    kernels = {n: s for n, s in segments("weight_grad.hip").items() if "weight_grad_kernel" in n and "join" not in n}
    assert len(kernels) == 4
    for name, parts in kernels.items():
        # the four steps of the loop: a thread's two loads to LDS, then its codes and their exponent byte
        assert sum(p == "LLrr" for p in parts) >= 4, (name, parts)
        for p in parts[:-1]:  # the last is the epilogue
            assert "rL" not in p, (name, parts)
