"""Which rows and keys the attention kernels touch, on the host: the header that finds them
(csrc/attention_sequences.h) is compiled into a program whose 64 lanes meet at every exchange
(tests/attention_sequences_check.cpp).  Whatever cu_q, cu_k and k_lens hold, every row of q, key and slot
of the workspace is inside its operand; where they ascend, each has its place once."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("attention") / "check")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{rocm}/include", f"-I{ROOT}/include",
                    f"-I{ROOT}/invariant_matmul_amd/csrc", "-o", out, f"{ROOT}/tests/attention_sequences_check.cpp"], check=True)
    return out


def check(program, q_rows, k_rows, heads, max_q, cu_q, cu_k, lens=(), causal=True, modes=("rows", "sorted", "keys", "chunks")):
    for mode in modes:
        if mode == "sorted" and len(cu_q) + 1 > 32:
            continue  # (up to 32 segments)
        args = [program, mode, q_rows, k_rows, *heads, max_q, int(causal), *cu_q, "--", *cu_k, "--", *lens]
        r = subprocess.run([str(x) for x in args], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, (mode, r.stdout, r.stderr)


def starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


@pytest.mark.parametrize("heads", [(4, 2), (1, 1), (100, 1)])
@pytest.mark.parametrize("lengths", [[1], [300], [5, 0, 7], [255, 1, 257], [130, 600, 0, 0, 3], [0]])
def test_sequences_have_their_places(program, lengths, heads):
    cu = starts(lengths)
    check(program, cu[-1], cu[-1], heads, max(1, max(lengths)), cu, cu)
    # a gap before, behind and, in the keys, lengths of their own
    rows = cu[-1] + 20
    check(program, rows, rows, heads, max(1, max(lengths)), [7 + x for x in cu], [9 + x for x in cu], [n // 2 for n in lengths])


@pytest.mark.parametrize("count", [29, 31, 61, 62, 63, 64, 127, 300, 4200])
def test_many_sequences_have_their_places(program, count):
    rng = random.Random(count)
    cu = starts([rng.choice([0, 1, 2, 3, 40 if count < 400 else 1]) for _ in range(count)])
    modes = ("rows", "sorted", "keys", "chunks") if count < 400 else ("rows",)
    check(program, cu[-1], cu[-1], (2, 1), 40, cu, cu, modes=modes)


# values that do not ascend, pass the operands or are negative
BAD = [([0, 90, 40], [0, 10, 1000], [5, 5000]), ([-5, 60, 50], [70, -3, 60], [-1, 9]),
       ([30, 10, BIG], [0, BIG, -BIG - 1], [BIG, BIG]), ([0, BIG, 0], [0, BIG, 0], [BIG, -BIG - 1]),
       ([0, 1000, 5], [0, 0, 900], [BIG, BIG]), ([1000, 500, 0], [1000, 500, 0], [BIG, BIG]), ([BIG, BIG, BIG], [BIG] * 3, [7, 7]),
       ([700, 0, 700], [0, 700, 0], [BIG, BIG])]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("arrays", BAD, ids=str)
def test_contents_of_the_arrays_stay_inside(program, arrays, causal):
    for (q_rows, k_rows), heads, max_q in (((1000, 1000), (4, 2), 3), ((50, 6000), (2, 1), 3), ((0, 100), (1, 1), 1), ((300, 0), (6, 2), 300)):
        check(program, q_rows, k_rows, heads, max_q, *arrays, causal=causal)


@pytest.mark.parametrize("seed", range(24))
def test_random_contents_stay_inside(program, seed):
    rng = random.Random(seed)
    count = rng.choice([1, 2, 5, 30, 62, 63, 64, 90])
    q_rows, k_rows = rng.choice([1, 60, 400]), rng.choice([1, 300, 1500])

    def draw(rows, n):
        return [rng.choice([rng.randint(0, rows), rng.randint(-5, rows + 5), rng.randint(-BIG - 1, BIG)]) for _ in range(n)]

    check(program, q_rows, k_rows, rng.choice([(4, 2), (3, 1), (70, 1)]), rng.choice([1, 3, q_rows]), draw(q_rows, count + 1),
          draw(k_rows, count + 1), draw(k_rows, count), causal=rng.random() < 0.7)
