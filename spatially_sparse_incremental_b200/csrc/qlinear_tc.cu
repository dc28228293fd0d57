#include "qlinear.cuh"
namespace sige {
bool qlinear_tc_scope(int) { return false; }
}
