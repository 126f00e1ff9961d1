"""The vocabulary operators' workspace holds what every call puts into it: sizes
counted on the host, from the library's own rules, without a device."""

import os
import random
import subprocess

import pytest

from tp_vocab_logits_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def count(tmp_path_factory):
    """count(configurations, embed): the numbers tests/vocab_sizes.cu prints."""
    folder = tmp_path_factory.mktemp("vocab_sizes")
    made = {}

    def run(configs, embed=False):
        if embed not in made:
            exe = str(folder / f"sizes_{int(embed)}")
            # Only its host code runs: the device code stays PTX.
            subprocess.run([_build.nvcc(), "-gencode", "arch=compute_103a,code=compute_103a",
                            "-std=c++17", f"-I{_build.INCLUDE}", f"-I{_build.CSRC}",
                            *(["-DEMBED"] if embed else []),
                            os.path.join(HERE, "vocab_sizes.cu"), "-o", exe], check=True)
            made[embed] = exe
        text = "\n".join(" ".join(map(str, c)) for c in configs)
        out = subprocess.run([made[embed]], input=text, capture_output=True, text=True, check=True)
        return [list(map(int, line.split())) for line in out.stdout.splitlines()]

    return run


# tp, W, K, max_rows, piece_cols, SMs: max_rows * tp passes 2^31.
BEYOND_INT = [(32, 1, 8, 1 << 26, 256, 152),
              (16, 100, 8, 1 << 27, 256, 152),
              (32, 2000, 8, (1 << 26) + 12345, 256, 152),
              (2, 1, 8, (1 << 30) - 1, 256, 152),
              (32, 1 << 24, 8, (1 << 30) - 1, 256, 152)]


def test_statistics_of_row_counts_beyond_32_bits(count):
    for config, (held, need, _, _) in zip(BEYOND_INT, count(BEYOND_INT)):
        tp, W, _, rows = config[:4]
        # Two halves of each vocabulary tile of at most 256 columns, for every row.
        assert need >= rows * 2 * tp * -(-W // 256)
        assert held >= need, config


def random_configs(seed, n, most_rows):
    r = random.Random(seed)

    def log_int(lo, hi):
        return max(lo, min(hi, round(lo * (hi / lo) ** r.random())))

    out = []
    for _ in range(n):
        W = log_int(1, 40000)
        whole = -(-W // 256) * 256
        out.append((r.choice([1, 2, 3, 8, 16, 32]), W, 8 * log_int(1, 1100), log_int(1, most_rows),
                    r.choice([256, whole, min(whole, 256 * log_int(1, 100))]),
                    r.choice([152, 148, 132])))
    return out


def test_every_call_fits(count):
    configs = random_configs(1, 150, 20000)
    got = count(configs)
    assert len(got) == len(configs)
    for config, (held, need, rows_held, rows_need) in zip(configs, got):
        assert held >= need, config
        assert rows_held >= rows_need, config


def test_every_lookup_gradient_fits(count):
    configs = random_configs(2, 300, 200000)
    got = count(configs, embed=True)
    assert len(got) == len(configs)
    for config, (held, need) in zip(configs, got):
        assert held >= need, config
