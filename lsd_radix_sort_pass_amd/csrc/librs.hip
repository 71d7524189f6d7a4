// librs.hip -- the library's translation unit: the sorts, and the
// mixture-of-experts calls, which use the sorts' launch, timing and argument
// helpers.
#include "rs.hip"

#include "experts.hip"
