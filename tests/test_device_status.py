"""How the kernels' status words become the one that the caller reads."""
import itertools
import os
import shutil
import subprocess

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nystr_coreset_approximate_b200", "csrc",
                      "device_status.h")
PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "%s"
int main(int n, char** words) {
    int code = 0;
    for (int k = 1; k < n; ++k)
        code = wildcat::graver_device_status(code, wildcat::device_status_code(atoi(words[k])));
    printf("%%d", code);
}
"""


def test_no_word_passes_for_success_and_the_gravest_wins(tmp_path):
    source, program = tmp_path / "status.cpp", str(tmp_path / "status")
    source.write_text(PROGRAM % HEADER)
    subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-o", program, str(source)], check=True, timeout=120)

    def code(*words):
        return int(subprocess.run([program, *map(str, words)], check=True, capture_output=True, text=True, timeout=60).stdout)

    assert code() == 0 and code(0, 0, 0) == 0
    for words, want in (((5,), 5), ((1,), 1), ((3,), 3), ((2,), 3), ((4,), 3), ((6,), 3), ((5, 3, 1), 5), ((3, 1), 3), ((6, 5), 5), ((6, 1), 3), ((1, 0), 1)):
        for order in itertools.permutations(words):
            assert code(*order) == want, order

