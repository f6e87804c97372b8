"""The two-word exp and ln of csrc_logits/tp_logits_two.cuh, compiled as host code (tests/host/two_check.cpp), against long
double. CPU only.

Bounds, from the roundings of words of at most 2^-6 (half a step: 2^-31 below 2^-7, 2^-30 above):
  exp, relative: the reduced argument's two (|r| <= ln 2/64), the polynomial's one, the product with the table's word one and
  a half: 4.5 x 2^-31 = 2.1e-9. Below e^-70 the second word loses bits under fp32's smallest step: at worst all of it, 2^-24.
  ln, absolute: the argument's two and the polynomial's one at 2^-31, the low words' two additions at 2^-30 each, the words of
  ln 2 127 x 2^-38: 7 x 2^-31 + 2^-31 = 3.7e-9."""
import os
import subprocess

from lazy_score_matrix_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_exp_and_ln_in_two_words(tmp_path):
    exe = str(tmp_path / "two_check")
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-w", "-isystem", cuda, "-I" + build.CSRC_LOGITS, "-o", exe,
                    os.path.join(HERE, "host", "two_check.cpp")], check=True, capture_output=True, text=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120).stdout.split()
    exp_normal, exp_low, ln, words = (float(v) for v in out[:4])
    print(out)
    assert exp_normal <= 2.2e-9 and exp_low <= 2.0 ** -24 and ln <= 3.7e-9
    assert words <= 2.0 ** -24 and out[4] == "1"  # |l| at most half a step of h
